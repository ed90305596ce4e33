// expert_ptx.cuh -- thin wrappers over the PTX the expert products use:
// mbarriers with bounded waits, TMA tile loads, and the 5th-generation tensor
// core instructions (tcgen05) with their shared-memory and instruction
// descriptors. Device code only.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "moe_ep.h"

namespace moe {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

// ---- mbarriers ------------------------------------------------------------
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

// "Elected" wrappers are called by a whole converged warp, with the same
// arguments in every lane; one lane (always the same) executes them. Written
// this way, and not inside a branch of one lane, the warp's loop keeps its
// addresses and descriptors in uniform registers.
__device__ __forceinline__ void mbar_expect_elected(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes)
      : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Without suspending the thread.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Address of this CTA's shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
  return r;
}
// A value at an address from cluster_addr.
__device__ __forceinline__ float ld_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// All threads of the cluster meet. The barrier's aligned forms are undefined unless a warp's
// lanes arrive together, which they need not do after a branch.
__device__ __forceinline__ void cluster_sync() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Arrivals on a barrier of the cluster (an address from cluster_addr). The
// relaxed forms order no memory: a release at cluster scope is a memory
// barrier that waits for the thread's stores (measured: one per stage halved
// the speed of the paired products). They serve where nothing is written for
// the other side: announcing copies, and handing back an accumulator whose
// loads tcgen05.wait::ld and tcgen05.fence have ordered.
__device__ __forceinline__ void mbar_arrive_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void mbar_expect_relaxed_elected(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "@q mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;\n\t}" ::"r"(
          bar),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_release(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}

// What a wait needs to give up: the CTA's abort flag (and its address in the
// other CTA of a pair, or 0), the clock cycles a wait may last, and the device
// status word.
struct WaitCtl {
  volatile int* abort;
  uint32_t peer_abort;
  long long limit;
  uint32_t* status;
};

// Waits for the phase of the given parity. False when the wait lasted longer
// than the limit (then the status bit is set and every other wait of the CTA
// or the pair gives up too) or another wait gave up.
template <bool PAIR>
__device__ __forceinline__ bool mbar_wait_slow(uint32_t bar, uint32_t parity, const WaitCtl& c) {
  const long long t0 = clock64();
  while (true) {
    if (*c.abort) return false;
    if (clock64() - t0 >= c.limit) {
      *c.abort = 1;
      if constexpr (PAIR)
        asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], %1;" ::"r"(c.peer_abort), "r"(1)
                     : "memory");
      atomicOr(c.status, MOE_STATUS_TIMEOUT);
      return false;
    }
    if (mbar_try(bar, parity)) return true;
  }
}

template <bool PAIR>
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, const WaitCtl& c) {
  if (mbar_test(bar, parity)) return true;
  if (c.limit > 0 && mbar_try(bar, parity)) return true;  // suspended for a while
  return mbar_wait_slow<PAIR>(bar, parity, c);
}

// Waits for copies or products in flight, abort flag or not, for at most about
// half a millisecond: the way out of a kernel, where they have landed unless a
// wait gave up.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try(bar, parity))
    if (clock64() - t0 > (1ll << 20)) return;
}

// ---- TMA ------------------------------------------------------------------
// Elected copies of a tile. CG == 2: `bar` is an address in the cluster, in
// either CTA of the pair.
#define MOE_TMA(DIM, GROUP, COORDS, ...)                                                          \
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"                           \
               "@q cp.async.bulk.tensor." DIM GROUP                                               \
               ".shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, " COORDS     \
               "], [%2];\n\t}" ::"r"(dst),                                                        \
               "l"(m), "r"(bar), __VA_ARGS__                                                      \
               : "memory")

template <int CG>
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x,
                                            int y) {
  if constexpr (CG == 2) MOE_TMA("2d", ".cta_group::2", "{%3, %4}", "r"(x), "r"(y));
  else MOE_TMA("2d", "", "{%3, %4}", "r"(x), "r"(y));
}

template <int CG>
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x,
                                            int y, int z) {
  if constexpr (CG == 2) MOE_TMA("3d", ".cta_group::2", "{%3, %4, %5}", "r"(x), "r"(y), "r"(z));
  else MOE_TMA("3d", "", "{%3, %4, %5}", "r"(x), "r"(y), "r"(z));
}
#undef MOE_TMA

__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}

// Orders shared-memory writes of this thread before later accesses of the
// asynchronous proxy (TMA, tensor cores).
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Copies of a tile from shared memory, of one group of the calling thread.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* m, uint32_t from, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];" ::
                   "l"(m),
               "r"(from), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, uint32_t from, int x, int y,
                                             int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          m),
      "r"(from), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Until the thread's copies have read their source, or are done.
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// ---- tcgen05 --------------------------------------------------------------
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// Whole warp; CG == 2: one warp of each CTA of the pair. 512 columns: the
// CTA's shared memory keeps any second CTA of these kernels off the SM, so the
// allocation never waits for one.
template <int CG>
__device__ __forceinline__ void tc_alloc(uint32_t smem_dst, uint32_t cols) {
  if constexpr (CG == 2) {
    asm volatile(
        "tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst),
        "r"(cols)
        : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  } else {
    asm volatile(
        "tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_dst),
        "r"(cols)
        : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
}

template <int CG>
__device__ __forceinline__ void tc_dealloc(uint32_t tmem, uint32_t cols) {
  if constexpr (CG == 2)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
  else
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(cols));
}

// Elected. The barrier (CG == 2: the barriers at this offset in both CTAs)
// gets an arrival when every product that the elected lane has issued so far
// is done (with an implied fence::before_thread_sync).
template <int CG>
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  if constexpr (CG == 2)
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster."
        "b64 [%0], %1;\n\t}" ::"r"(bar),
        "h"((uint16_t)3)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            bar)
        : "memory");
}

// Elected. N products (1 or 2) along the reduction axis, the second with both
// descriptors advanced; `accumulate`: the first adds to the accumulator (a
// second always does).
#define MOE_TC_MMA(GROUP, KIND, SECOND)                                                            \
  asm volatile("{\n\t.reg .pred p, t, q;\n\t.reg .b64 a, b;\n\t"                                  \
               "elect.sync _|q, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"                          \
               "setp.eq.b32 t, 0, 0;\n\tadd.u64 a, %1, %5;\n\tadd.u64 b, %2, %6;\n\t"              \
               "@q tcgen05.mma.cta_group::" GROUP ".kind::" KIND " [%0], %1, %2, %3, p;\n\t"      \
               SECOND "\n\t}" ::"r"(d),                                                            \
               "l"(da), "l"(db), "r"(idesc), "r"((uint32_t)accumulate), "l"(step_a), "l"(step_b)   \
               : "memory")
#define MOE_TC_MMA_N(GROUP, KIND)                                                                  \
  do {                                                                                             \
    if constexpr (N == 2)                                                                          \
      MOE_TC_MMA(GROUP, KIND, "@q tcgen05.mma.cta_group::" GROUP ".kind::" KIND                    \
                              " [%0], a, b, %3, t;");                                              \
    else                                                                                           \
      MOE_TC_MMA(GROUP, KIND, "");                                                                 \
  } while (0)

template <int CG, bool FP8, int N>
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t da, uint64_t db, uint64_t step_a,
                                       uint64_t step_b, uint32_t idesc, bool accumulate) {
  if constexpr (CG == 2 && FP8) MOE_TC_MMA_N("2", "f8f6f4");
  else if constexpr (CG == 2) MOE_TC_MMA_N("2", "f16");
  else if constexpr (FP8) MOE_TC_MMA_N("1", "f8f6f4");
  else MOE_TC_MMA_N("1", "f16");
}
#undef MOE_TC_MMA_N
#undef MOE_TC_MMA

// 32 consecutive columns of this warp's 32 lanes: v[i] = column i of the
// thread's lane. Asynchronous until tc_wait_ld.
__device__ __forceinline__ void tc_ld32(uint32_t (&v)[32], uint32_t taddr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]),
        "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
        "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tc_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Ties the loaded registers to this place: their uses stay after the wait
// that precedes it.
__device__ __forceinline__ void tc_loaded(uint32_t (&v)[32]) {
  asm volatile(""
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]),
                 "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]), "+r"(v[9]),
                 "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]),
                 "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]),
                 "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]),
                 "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31]));
}

// 16 consecutive columns of this warp's 32 lanes: column i of the thread's lane
// = v[i]. Asynchronous until tc_wait_st.
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
      "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Elected. One product of 16 k with A in tensor memory (fp16, two k a column).
__device__ __forceinline__ void tc_mma_ta(uint32_t d, uint32_t a, uint64_t db, uint32_t idesc,
                                          bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\telect.sync _|q, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(db), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

// Shared-memory descriptor of an operand tile with 128-byte swizzled rows.
// K-major (lbo unused): rows of 128 bytes along K, 8-row groups sbo apart.
// MN-major: lines of 128 bytes along M or N, one per k, groups of 8 k sbo
// apart, and the next 128 bytes along M or N lbo apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) |
         ((uint64_t)(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// Instruction descriptor: fp32 accumulator, A and B of one type (bf16; or the
// first of the kind, e4m3 of f8f6f4 and fp16 of f16), their majors, M and N.
__host__ __device__ constexpr uint32_t mma_desc(bool fp8, bool a_mn, bool b_mn, int M, int N) {
  return (1u << 4) | (fp8 ? 0u : (1u << 7) | (1u << 10)) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

}  // namespace moe
