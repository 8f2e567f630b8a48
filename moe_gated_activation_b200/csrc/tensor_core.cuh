// sm_100a tensor-core (tcgen05), cluster and TMA wrappers of the grouped
// products.  CG: the SMs that work on one tile (cta_group::1 or ::2).
#pragma once

#include "device_common.cuh"

namespace moeact {
namespace tc {

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* dst, uint32_t ncols) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_addr(dst)), "r"(ncols) : "memory");
  else
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_addr(dst)), "r"(ncols) : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_relinquish() {
  if constexpr (CG == 1)
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  else
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// Arrives on `bar` -- with CG = 2 on the barrier at that offset in both SMs of
// the pair -- once every tcgen05 operation this thread issued has completed.
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 ::"r"(smem_addr(bar)) : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_addr(bar)), "h"((uint16_t)3) : "memory");
}
// D (+)= A x B^T, both operands with E8M0 scales of 32 values: F4 = false: 32
// E4M3 values of the summed index, F4 = true: 64 E2M1 values.
template <int CG, bool F4>
__device__ __forceinline__ void mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                    uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
#define MOEACT_MMA(KIND)                                                                     \
  asm volatile("{ .reg .pred p; setp.ne.b32 p, %4, 0; " KIND " [%0], %1, %2, %3, [%5], [%6], " \
               "p; }" ::"r"(d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(sfa),  \
               "r"(sfb)                                                                        \
               : "memory")
  if constexpr (CG == 1 && !F4) MOEACT_MMA("tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale");
  if constexpr (CG == 2 && !F4) MOEACT_MMA("tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale");
  if constexpr (CG == 1 && F4)
    MOEACT_MMA("tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X");
  if constexpr (CG == 2 && F4)
    MOEACT_MMA("tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X");
#undef MOEACT_MMA
}
// One or four 32-bit words into consecutive columns of the warp's 32 lanes.
__device__ __forceinline__ void st1(uint32_t taddr, uint32_t v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(v)
               : "memory");
}
__device__ __forceinline__ void st4(uint32_t taddr, uint32_t v0, uint32_t v1, uint32_t v2,
                                    uint32_t v3) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};"
               ::"r"(taddr), "r"(v0), "r"(v1), "r"(v2), "r"(v3) : "memory");
}
__device__ __forceinline__ void wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 32 consecutive columns of the warp's 32 lanes (thread t: lane t).
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]),
        "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]),
        "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]),
        "=r"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// No use of what a load brought (32 registers) moves up past this point.
__device__ __forceinline__ void tie(uint32_t* v) {
  asm volatile(""
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]),
                 "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                 "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]),
                 "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]),
                 "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]),
                 "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]),
                 "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}

// One lane of a converged warp, the same lane every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.aligned; barrier.cluster.wait.aligned;" ::: "memory");
}
// The cluster address, in the pair's first SM, of this SM's shared-memory
// object at `p`.
__device__ __forceinline__ uint32_t leader_addr(const void* p) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_addr(p)));
  return r;
}
__device__ __forceinline__ void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
// What an arrival on a barrier and the wait for it order.
enum Order : int {
  kSm,        // everything, between threads of one SM
  kPair,      // between the SMs of a pair, tensor memory only (fence_before before
              // the arrival, fence_after after the wait): no memory is handed over
  kPairData,  // a wait, between the SMs of a pair: also what their copies wrote
};

// An arrival on a barrier of the pair's first SM (bar: its cluster address).
template <Order O>
__device__ __forceinline__ void arrive_leader(uint32_t bar) {
  if constexpr (O == kSm)
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
  else
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
                 : "memory");
}
__device__ __forceinline__ void arrive_tx(uint32_t bar, uint32_t bytes) {   // this SM's
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void arrive_tx_leader(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;"
               ::"r"(bar), "r"(bytes) : "memory");
}
// 2-D tile load into this SM's shared memory, completing on the barrier at
// cluster address `bar` (this SM's, or with CG = 2 the pair's first SM's).
template <int CG>
__device__ __forceinline__ void load_2d(void* dst, const void* tmap, int x, int y, uint32_t bar) {
  if constexpr (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::"
        "bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_addr(dst)), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void prefetch_map(const void* tmap) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tmap)) : "memory");
}

// Bulk tensor stores from shared memory and (add_*: fp32, rounded to nearest,
// subnormals kept: held to by the tests) additions to what the output holds;
// bulk_wait_read: the ones committed have read their shared memory, bulk_wait:
// they are done.
__device__ __forceinline__ void store_2d(const void* tmap, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];"
               ::"l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_addr(src)), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void store_3d(const void* tmap, const void* src, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];"
      ::"l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_addr(src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void add_2d(const void* tmap, const void* src, int x, int y) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];"
      ::"l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_addr(src)), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void add_3d(const void* tmap, const void* src, int x, int y, int z) {
  asm volatile(
      "cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], "
      "[%1];"
      ::"l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_addr(src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Bounded waits (the global timer, one second).  spin: without suspending,
// for the single warps that feed the tensor cores, whose wake-up latency
// counts.
#define MOEACT_WAIT_ASM(FORM, SCOPE, HINT)                                               \
  asm volatile("{ .reg .pred p; " FORM SCOPE "shared::cta.b64 p, [%1], %2" HINT          \
               "; selp.u32 %0, 1, 0, p; }"                                               \
               : "=r"(ok) : "r"(smem_addr(bar)), "r"(parity), "r"(kWaitHintNs) : "memory")
#define MOEACT_WAIT_FORM(NAME, FORM, HINT)                                               \
  template <Order O>                                                                     \
  __device__ __forceinline__ bool NAME(uint64_t* bar, uint32_t parity) {                 \
    uint32_t ok;                                                                         \
    if constexpr (O == kSm) MOEACT_WAIT_ASM(FORM, "", HINT);                             \
    else if constexpr (O == kPair) MOEACT_WAIT_ASM(FORM, "relaxed.cluster.", HINT);      \
    else MOEACT_WAIT_ASM(FORM, "acquire.cluster.", HINT);                                \
    return ok != 0;                                                                      \
  }
MOEACT_WAIT_FORM(test, "mbarrier.test_wait.parity.", "")
MOEACT_WAIT_FORM(test_sleep, "mbarrier.try_wait.parity.", ", %3")
#undef MOEACT_WAIT_FORM
#undef MOEACT_WAIT_ASM
template <Order O>
__device__ __forceinline__ bool spin(uint64_t* bar, uint32_t parity) {
  if (test<O>(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (;;) {
    for (int i = 0; i < 64; ++i)
      if (test<O>(bar, parity)) return true;
    if (global_ns() - t0 > kWaitLimitNs) return false;
  }
}
template <Order O>
__device__ __forceinline__ bool sleep(uint64_t* bar, uint32_t parity) {
  if (test_sleep<O>(bar, parity)) return true;
  const uint64_t t0 = global_ns();
  for (;;) {
    for (int i = 0; i < 4; ++i)
      if (test_sleep<O>(bar, parity)) return true;
    if (global_ns() - t0 > kWaitLimitNs) return false;
  }
}

__device__ __forceinline__ void fence_proxy_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Shared-memory descriptor of an operand tile of 128-byte rows in the 128-byte
// swizzled layout (16-byte chunk c of row r at c ^ (r mod 8), 8-row groups
// 1024 bytes apart; descriptor version 1).  Rows are those of the output
// (the summed index inside a row), or, with the major bit of the instruction
// descriptor set, of the summed index.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

}  // namespace tc
}  // namespace moeact
