// Pieces shared by the latent attention kernels: waits of a whole warp, tensor
// memory accesses, descriptors of operands that lie with their M or N dimension
// contiguous.
#pragma once

#include <cuda.h>

#include <cmath>

#include "moe_fp4_internal.cuh"
#include "mxfp4_ops.cuh"
#include "ptx_sm103.cuh"
#include "tc_helpers.cuh"

namespace moe_fp4 {
namespace latent {

constexpr int kSmemMax = 227 * 1024;
constexpr int kLatent = 512, kRope = 64, kRow = kLatent + kRope;  // of a cached token
constexpr int kNope = 128, kValue = 128;                          // of an expanded head

// a value that is the same in all lanes, in a form that lets the compiler know it
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }

// true in one lane of the (converged) warp; the tensor-core and TMA instructions
// issued under it take their operands from uniform registers
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

struct Waits {
  volatile int* abort_flag;
  int32_t* err;
  uint64_t limit_ns;
  // a bounded wait of the whole (converged) warp
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) const {
    if (__all_sync(0xFFFFFFFFu, mbar_try_wait(bar, parity))) return true;
    // (mbar_wait in fewer instructions: the kernels wait in many places, and are near what the instruction cache holds)
    const uint64_t since = global_timer_ns();
    bool ok;
    do
      ok = mbar_try_wait_sleep(bar, parity);
    while (!ok && !*abort_flag && global_timer_ns() - since <= limit_ns);
    if (!ok) {
      *abort_flag = 1;
      atomicOr(err, kErrWaitTimeout);
    }
    return __all_sync(0xFFFFFFFFu, ok);
  }
  __device__ __forceinline__ void drain(uint64_t* bar, uint32_t parity) const {
    mbar_wait_drain(bar, parity, err, kErrWaitTimeout, limit_ns);
  }
};

// whether the phase has completed, without waiting; the same in all lanes
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return __all_sync(0xFFFFFFFFu, ok != 0);
}

// Shared-memory descriptors, 128-byte swizzle, as two words (the low one holds the
// address).  K-major: rows of 128 bytes (64 elements of K), groups of 8 rows 1 KB
// apart.  MN-major: rows of 128 bytes are 64 elements of M or N for one element of
// K, groups of 8 K 1 KB apart, the next 64 elements of M or N `pitch` bytes on.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t pitch) {
  return ((saddr & 0x3FFFFu) >> 4) | ((pitch >> 4) << 16);
}
__device__ __forceinline__ uint64_t desc(uint32_t lo) { return ((uint64_t)kDescHi << 32) | lo; }

// bf16 operands, fp32 sums; a_mn / b_mn: the operand is MN-major
__device__ __forceinline__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}

// D[tmem] (+)= A[smem] B[smem]
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// this thread's lane, 32 columns; valid after tmem_wait_ld
__device__ __forceinline__ void tmem_ld32(uint32_t ta, uint32_t (&a)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
        "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]),
        "=r"(a[16]), "=r"(a[17]), "=r"(a[18]), "=r"(a[19]), "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]),
        "=r"(a[24]), "=r"(a[25]), "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31])
      : "r"(ta)
      : "memory");
}

// 16 lanes by 64 columns of 32 bits, as fragments: a[4 i + 2 r + j] is row lane / 4
// + 8 r, column 8 i + 2 (lane % 4) + j
__device__ __forceinline__ void tmem_ld_rows16(uint32_t ta, uint32_t (&a)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
        "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15]),
        "=r"(a[16]), "=r"(a[17]), "=r"(a[18]), "=r"(a[19]), "=r"(a[20]), "=r"(a[21]), "=r"(a[22]), "=r"(a[23]),
        "=r"(a[24]), "=r"(a[25]), "=r"(a[26]), "=r"(a[27]), "=r"(a[28]), "=r"(a[29]), "=r"(a[30]), "=r"(a[31])
      : "r"(ta)
      : "memory");
}

// the same of 32 columns
__device__ __forceinline__ void tmem_ld_rows16_half(uint32_t ta, uint32_t* a) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]),
        "=r"(a[8]), "=r"(a[9]), "=r"(a[10]), "=r"(a[11]), "=r"(a[12]), "=r"(a[13]), "=r"(a[14]), "=r"(a[15])
      : "r"(ta)
      : "memory");
}

// four 8 x 8 matrices of 16 bits, fragments as of mma, stored transposed: lane 8 k +
// c gives the address of the 16 bytes of matrix k's column c
__device__ __forceinline__ void stmatrix4_trans(void* p, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(smem_u32(p)), "r"(a), "r"(b),
               "r"(c), "r"(d)
               : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// the same bytes to L2 only
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(z) : "memory");
}

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(smem_u32(dst)),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// whether the predicate holds in any of the `threads` threads at barrier `id`;
// the barrier has no time limit: all of them come to every one of its uses
__device__ __forceinline__ bool any_at_barrier(bool v, int id, int threads) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred pin, pout;\n\tsetp.ne.u32 pin, %1, 0;\n\tbar.red.or.pred pout, %3, %2, pin;\n\t"
      "selp.u32 %0, 1, 0, pout;\n}"
      : "=r"(any)
      : "r"(v ? 1u : 0u), "r"(threads), "r"(id)
      : "memory");
  return any != 0;
}

}  // namespace latent

constexpr int kMaxSequences = 1 << 24;  // every CTA looks through them
// the scale, and its multiple that exp2 takes
inline bool finite_scale(float scale) { return std::isfinite(scale * 1.4426950408889634f); }

bool make_map_3d(CUtensorMap* m, const void* base, const uint64_t (&dims)[3], const uint64_t (&strides)[2],
                 const uint32_t (&box)[3]);  // bf16, 128-byte swizzle

}  // namespace moe_fp4
