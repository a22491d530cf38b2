// sm_100a building blocks of the prompt attention kernels: bounded mbarrier
// waits, TMA tile loads, tcgen05 matrix instructions and TMEM access.
#pragma once

#include <cuda.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kvq_device.cuh"

namespace kvq {
namespace sm100 {

constexpr long long kWaitLimitNs = 2000000000LL;  // bounded waits: 2 s

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// true in one lane of the (converged) warp
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(r));
  return r != 0;
}

// ---- mbarriers
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_init_fence() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, "
      "p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ long long global_ns() {
  long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// arrive from the lane where `who` is set, without a branch
__device__ __forceinline__ void mbar_arrive_if(bool who, uint32_t bar) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %1, 0;\n @p mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n}" ::"r"(
          bar),
      "r"(static_cast<uint32_t>(who))
      : "memory");
}
// Wait for a phase; false once the limit passes or `stop` (shared memory, set
// by whichever warp of the CTA gave up first) is set.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int* stop) {
  if (mbar_try(bar, parity)) return true;
  const long long t0 = global_ns();
  while (!mbar_try(bar, parity)) {
    if (*stop) return false;
    if (global_ns() - t0 > kWaitLimitNs) {
      *stop = 1;
      return false;
    }
  }
  return true;
}

// The same by a whole warp, with one answer for its lanes (the common case is
// one try and one vote).
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* stop) {
  if (__all_sync(kFull, mbar_try(bar, parity))) return true;
  return __all_sync(kFull, mbar_wait(bar, parity, stop));
}

// ---- TMA: one box of a 3-D map (channel, head, row)
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int channel, int head, int row,
                                         uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(channel), "r"(head), "r"(row), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// generic-proxy writes to shared memory before async-proxy (TMA, MMA) accesses
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---- tcgen05
// Shared-memory matrix descriptor, 128-byte swizzle, 64-element (128-byte)
// rows in groups of eight (1024 bytes).  K-major operands (Q, K): `lead` is
// unused; the 8-row groups follow one another.  MN-major operands (V: keys as
// rows, channels contiguous): `lead` is the distance of the next 64 channels,
// and the 8-key groups follow one another.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr, uint32_t lead) {
  uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFF);
  d |= static_cast<uint64_t>((lead >> 4) & 0x3FFF) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;  // descriptor version
  d |= static_cast<uint64_t>(2) << 61;  // 128-byte swizzle
  return d;
}
// kind::f16 instruction descriptor: fp32 accumulators, fp16 A (K-major) and
// B, M = 128; b_mn: B is MN-major
__host__ __device__ constexpr uint32_t idesc_m128(uint32_t n, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(
          d),
      "l"(da), "l"(db), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}
// A from TMEM: one row per lane, fp16 pairs, 8 columns per 16 elements
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t db, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(
          d),
      "r"(a), "l"(db), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}
// arrive at `bar` when every MMA this thread issued so far has finished
__device__ __forceinline__ void mma_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_alloc512(uint32_t slot) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(slot) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free512(uint32_t base) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(base));
}

// 32 consecutive 32-bit columns of this thread's TMEM lane; not yet waited for
#define KVQ_R32(r, o)                                                                                             \
  "=f"(r[o]), "=f"(r[o + 1]), "=f"(r[o + 2]), "=f"(r[o + 3]), "=f"(r[o + 4]), "=f"(r[o + 5]), "=f"(r[o + 6]),     \
      "=f"(r[o + 7]), "=f"(r[o + 8]), "=f"(r[o + 9]), "=f"(r[o + 10]), "=f"(r[o + 11]), "=f"(r[o + 12]),          \
      "=f"(r[o + 13]), "=f"(r[o + 14]), "=f"(r[o + 15]), "=f"(r[o + 16]), "=f"(r[o + 17]), "=f"(r[o + 18]),       \
      "=f"(r[o + 19]), "=f"(r[o + 20]), "=f"(r[o + 21]), "=f"(r[o + 22]), "=f"(r[o + 23]), "=f"(r[o + 24]),       \
      "=f"(r[o + 25]), "=f"(r[o + 26]), "=f"(r[o + 27]), "=f"(r[o + 28]), "=f"(r[o + 29]), "=f"(r[o + 30]),       \
      "=f"(r[o + 31])
#define KVQ_W32(r, o)                                                                                             \
  "+f"(r[o]), "+f"(r[o + 1]), "+f"(r[o + 2]), "+f"(r[o + 3]), "+f"(r[o + 4]), "+f"(r[o + 5]), "+f"(r[o + 6]),     \
      "+f"(r[o + 7]), "+f"(r[o + 8]), "+f"(r[o + 9]), "+f"(r[o + 10]), "+f"(r[o + 11]), "+f"(r[o + 12]),          \
      "+f"(r[o + 13]), "+f"(r[o + 14]), "+f"(r[o + 15]), "+f"(r[o + 16]), "+f"(r[o + 17]), "+f"(r[o + 18]),       \
      "+f"(r[o + 19]), "+f"(r[o + 20]), "+f"(r[o + 21]), "+f"(r[o + 22]), "+f"(r[o + 23]), "+f"(r[o + 24]),       \
      "+f"(r[o + 25]), "+f"(r[o + 26]), "+f"(r[o + 27]), "+f"(r[o + 28]), "+f"(r[o + 29]), "+f"(r[o + 30]),       \
      "+f"(r[o + 31])
template <int O, int N>
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float (&v)[N]) {
  static_assert(O + 32 <= N, "columns fit");
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%"
      "19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : KVQ_R32(v, O)
      : "r"(addr));
}
// wait for the loads above; ties the 32 registers to the wait
template <int O, int N>
__device__ __forceinline__ void tmem_wait32(float (&v)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : KVQ_W32(v, O));
}
// eight columns, loaded and waited for
__device__ __forceinline__ void tmem_ld8(uint32_t addr, float (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
               : "r"(addr));
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]));
}
__device__ __forceinline__ void tmem_st8(uint32_t addr, const float (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}
#undef KVQ_R32
#undef KVQ_W32
template <int O, int N>
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&v)[N]) {
  static_assert(O + 32 <= N, "columns fit");
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(v[O]), "r"(v[O + 1]), "r"(v[O + 2]), "r"(v[O + 3]), "r"(v[O + 4]), "r"(v[O + 5]), "r"(v[O + 6]),
      "r"(v[O + 7]), "r"(v[O + 8]), "r"(v[O + 9]), "r"(v[O + 10]), "r"(v[O + 11]), "r"(v[O + 12]), "r"(v[O + 13]),
      "r"(v[O + 14]), "r"(v[O + 15]), "r"(v[O + 16]), "r"(v[O + 17]), "r"(v[O + 18]), "r"(v[O + 19]),
      "r"(v[O + 20]), "r"(v[O + 21]), "r"(v[O + 22]), "r"(v[O + 23]), "r"(v[O + 24]), "r"(v[O + 25]),
      "r"(v[O + 26]), "r"(v[O + 27]), "r"(v[O + 28]), "r"(v[O + 29]), "r"(v[O + 30]), "r"(v[O + 31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 2^x (the hardware approximation; -inf gives 0)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace sm100
}  // namespace kvq
