// Inline-PTX wrappers for the tensor-core operators (sm_100a): tcgen05 matrix products with
// accumulators in tensor memory, tensor-map copies, and waits that end.
//
// Copies read this GPU's own memory into the issuing CTA's shared memory, without multicast.
#pragma once
#include <cuda.h>
#include <stdint.h>

#include "ptx.cuh"

namespace tre {
namespace tc {

// ---- bounded waits --------------------------------------------------------------------
// Every wait gives up after about two seconds, or at once when another role of the CTA has:
// it then sets the CTA's flag, and the caller leaves its loop for the common teardown.
constexpr long long kWaitClocks = 4000000000ll;

// A probe that may sleep up to a millisecond before it answers: a spinning warp would take
// issue slots from the warps that it waits for.
__device__ __forceinline__ bool try_wait_long(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, volatile int* gave_up,
                                     long long limit = kWaitClocks) {
  if (try_wait_long(bar, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (try_wait_long(bar, parity)) return true;
    if (*gave_up || clock64() - t0 > limit) {
      *gave_up = 1;
      return false;
    }
  }
}

// The same by a whole warp: every lane returns what all of them found.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* gave_up,
                                          long long limit = kWaitClocks) {
  return __all_sync(0xffffffffu, wait(bar, parity, gave_up, limit));
}

// What a CTA has issued ends before the CTA does: another role may give up after the issuing one
// has left its loop, so both are waited for whatever has happened, and nothing is lost by it where
// all went well (the sums that the CTA stores come after them).  Two seconds for all of them.
__device__ __forceinline__ void settle(uint64_t* bar, uint32_t parity, long long since) {
  while (!mbar_try_wait(bar, parity) && clock64() - since < kWaitClocks) {
  }
}

// `issued` copies over a ring of `places`: the last one of each place.
__device__ __forceinline__ void settle_copies(uint64_t* full, int issued, int places,
                                              long long since) {
  for (int i = max(0, issued - places); i < issued; ++i)
    settle(full + i % places, i / places & 1, since);
}

// ---- one lane of a converged warp -------------------------------------------------------
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// ---- registers and paired arithmetic -----------------------------------------------------
// By every warp of a warpgroup.  What the groups take must not exceed what the CTA was
// launched with (its threads times the registers of a thread).
template <int N>
__device__ __forceinline__ void regs_more() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_less() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Two fp32 operations of one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mov.b64 c, {%6, %7};\n\tfma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// ---- tensor-map copies -------------------------------------------------------------------
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

__device__ __forceinline__ void load_2d(void* dst, const CUtensorMap* m, int x, int y,
                                        uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(m), "r"(x), "r"(y), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void load_3d(void* dst, const CUtensorMap* m, int x, int y, int z,
                                        uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

// 16 bytes from global to shared memory by this thread, or zeros; the wait is for all of its own.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(there ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copy16_wait() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Makes this thread's writes to shared memory visible to the copy and matrix units.
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// ---- tensor memory -------------------------------------------------------------------------
// Whole warp; cols a power of two, 32 .. 512.  The address goes to shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                   smem_u32(dst)),
               "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols)
               : "memory");
}

// An address is lane << 16 | column; a warp reaches the 32 lanes 32 (warp mod 4) + lane.
#define TRE_R8(v, o)                                                                        \
  "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), \
      "=r"(v[o + 6]), "=r"(v[o + 7])
#define TRE_W8(v, o)                                                                       \
  "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]),      \
      "r"(v[o + 6]), "r"(v[o + 7])

__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t* v) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : TRE_R8(v, 0)
               : "r"(addr));
}

__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : TRE_R8(v, 0), TRE_R8(v, 8), TRE_R8(v, 16), TRE_R8(v, 24)
      : "r"(addr));
}

__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31, %32};" ::"r"(addr),
      TRE_W8(v, 0), TRE_W8(v, 8), TRE_W8(v, 16), TRE_W8(v, 24)
      : "memory");
}
#undef TRE_R8
#undef TRE_W8

__device__ __forceinline__ void wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// Order tensor-memory work around a barrier between threads: before the arrival, after the
// wait.
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// ---- matrix products ----------------------------------------------------------------------
// Instruction word of kind::f16 with bf16 operands and fp32 sums: M x N, A with k running
// fastest, B with k fastest (b_mn 0) or with n fastest (b_mn 1).
__host__ __device__ constexpr uint32_t idesc_bf16(uint32_t m, uint32_t n, uint32_t b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_mn << 16) | ((n >> 3) << 17) | ((m >> 4) << 24);
}

// Shared-memory operand in rows of 128 bytes with the 128-byte swizzle (16-byte chunk c of row
// r sits at chunk c ^ (r mod 8)), tiles aligned to 1024 bytes.  `sbo`: bytes from 8 rows to
// the next 8; `lbo`: bytes from 64 elements along the rows to the next 64 (used when n runs
// fastest; ignored otherwise).
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3ffffu) >> 4) | ((uint64_t)(lbo >> 4) << 16) |
         ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// The same from its two halves: the upper is a constant of the layout, the lower moves by
// bytes / 16.
__device__ __forceinline__ constexpr uint32_t desc_hi(uint32_t sbo) {
  return (sbo >> 4) | (1u << 14) | (2u << 29);
}
__device__ __forceinline__ constexpr uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  return ((addr & 0x3ffffu) >> 4) | ((lbo >> 4) << 16);
}
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) {
  return (uint64_t)hi << 32 | lo;
}

// D (tensor memory) = or += A (shared) B (shared), by one thread.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

// The same with A in tensor memory (lane = row, two k per 32-bit column).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}

// Arrive on `bar` once every product this thread has issued so far is done.
__device__ __forceinline__ void commit(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_u32(bar))
      : "memory");
}

}  // namespace tc
}  // namespace tre
