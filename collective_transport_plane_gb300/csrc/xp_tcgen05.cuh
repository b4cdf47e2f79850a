// The fifth-generation tensor core's instructions, its memory (TMEM) and the
// tiled copies that feed it, as the product of 8-bit matrices uses them.
#pragma once

#include <cuda.h>

#include <cstdint>

namespace xp {
namespace tc {

__device__ __forceinline__ unsigned smem_of(const void* p) { return (unsigned)__cvta_generic_to_shared(p); }

// One lane of a converged warp, the same each time.  (Code that the warp walks
// through together with an elected lane's instructions in between keeps its
// values in uniform registers, which the tensor core's instructions take: a
// product's block of 128 columns took 800 cycles to issue from a lane's own loop.)
__device__ __forceinline__ bool elected() {
  unsigned p;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}

// ---- mbarriers, all waits with a limit
__device__ __forceinline__ void bar_init(unsigned bar, unsigned count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_expect(unsigned bar, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// What a copy that was never asked for would have counted.
__device__ __forceinline__ void bar_uncount(unsigned bar, unsigned bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// CLUSTER: what the arriving threads of other CTAs wrote before is seen.
template <bool CLUSTER>
__device__ __forceinline__ bool bar_try(unsigned bar, unsigned parity) {
  unsigned ok;
  if constexpr (CLUSTER)
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  else
    asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}"
                 : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// A wait gives up after `limit` ns of the GPU's clock, which it looks at after 64
// tries of up to 4 us each, or after each where the limit is below a millisecond.
// (No wait here is for another kernel, and the longest loop of products takes
// milliseconds.)
__device__ __forceinline__ unsigned long long clock_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
template <bool CLUSTER>
__device__ __noinline__ bool bar_wait_long(unsigned bar, unsigned parity, unsigned long long limit) {
  const unsigned long long start = clock_ns();
  const int tries = limit < 1000000 ? 1 : 64;
  do {
    for (int i = 0; i < tries; ++i)
      if (bar_try<CLUSTER>(bar, parity)) return true;
  } while (clock_ns() - start < limit);
  return false;
}
template <bool CLUSTER = false>
__device__ __forceinline__ bool bar_wait(unsigned bar, unsigned parity, unsigned long long limit) {
  return bar_try<CLUSTER>(bar, parity) || bar_wait_long<CLUSTER>(bar, parity, limit);
}

// The same without a call, for a function that is called itself.
__device__ __forceinline__ void bar_wait_here(unsigned bar, unsigned parity, unsigned long long limit) {
  for (const unsigned long long start = clock_ns(); !bar_try<false>(bar, parity) && clock_ns() - start < limit;) {
  }
}

// ---- the CTAs of a cluster
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
// Where a CTA's shared memory address lies in the cluster's.
__device__ __forceinline__ unsigned in_cta(unsigned smem, unsigned rank) {
  unsigned r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_in_cta(unsigned smem, unsigned rank, unsigned v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(in_cta(smem, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ unsigned load_in_cta(unsigned smem, unsigned rank) {
  unsigned v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(in_cta(smem, rank)) : "memory");
  return v;
}
__device__ __forceinline__ void bar_arrive_cluster(unsigned bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// One that publishes nothing in memory, and waits for no store before it.
__device__ __forceinline__ void bar_arrive_relaxed(unsigned bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// ---- tiled copies into shared memory
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
// The box of `m` whose first element is column x of row y.  CTAS 2: the barrier may be the other CTA's of a pair.
template <int CTAS>
__device__ __forceinline__ void load_box(unsigned smem, const CUtensorMap* m, int x, int y, unsigned bar) {
  if constexpr (CTAS == 1)
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(smem), "l"(m), "r"(x), "r"(y), "r"(bar) : "memory");
  else
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];"
                 ::"r"(smem), "l"(m), "r"(x), "r"(y), "r"(bar) : "memory");
}

// ---- TMEM: 128 lanes of 512 columns of 32 bits; an address is lane << 16 | column.
// CTAS 2: a warp of each CTA of a pair takes part.
template <int CTAS>
__device__ __forceinline__ void tmem_alloc(unsigned result_smem, unsigned columns) {
  if constexpr (CTAS == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(result_smem), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(result_smem), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
}
template <int CTAS>
__device__ __forceinline__ void tmem_free(unsigned at, unsigned columns) {
  if constexpr (CTAS == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}
// 16 columns of the warp's 32 lanes, a lane's into its own registers: there
// after tmem_wait() and landed() of them.
__device__ __forceinline__ void tmem_load16(unsigned at, float (&v)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
                 "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
               : "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// No use of the registers moves before this.
__device__ __forceinline__ void landed(float (&v)[16]) {
  asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]),
               "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---- operands in shared memory
// Rows of 128 bytes in groups of 8 (1024 bytes), swizzled over 128 bytes as the
// tiled copies write them.  32 bytes further along the rows is 2 more here.
__device__ __forceinline__ unsigned long long rows128(unsigned smem) {
  return (unsigned long long)(smem >> 4 & 0x3fff) | 1ull << 16 | 64ull << 32 | 1ull << 46 | 2ull << 61;
}
// Rows of 16 bytes, unswizzled, groups of 8 one behind another: scales.
__device__ __forceinline__ unsigned long long rows16(unsigned smem) {
  return (unsigned long long)(smem >> 4 & 0x3fff) | 8ull << 32 | 1ull << 46;
}
// 32 rows of 16 bytes to 4 columns, the same for each 32 lanes.  CTAS 2: in
// both CTAs of a pair, each from its own shared memory.
template <int CTAS>
__device__ __forceinline__ void copy_scales(unsigned tmem, unsigned long long rows) {
  if constexpr (CTAS == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(rows) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(rows) : "memory");
}
// d = [d +] a b^T over 32 columns of codes (e4m3), each row's 32 columns times
// the power of two that its scale byte says.  CTAS 2: 256 rows of a, half of
// them in each CTA's shared memory and TMEM, and half of b's rows in each's.
template <int CTAS>
__device__ __forceinline__ void mma_scaled(unsigned d, unsigned long long a, unsigned long long b, unsigned shape, unsigned scale_a,
                                           unsigned scale_b, bool add) {
  if constexpr (CTAS == 1)
    asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %6, 0;\n"
                 "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}"
                 ::"r"(d), "l"(a), "l"(b), "r"(shape), "r"(scale_a), "r"(scale_b), "r"((unsigned)add) : "memory");
  else
    asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %6, 0;\n"
                 "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}"
                 ::"r"(d), "l"(a), "l"(b), "r"(shape), "r"(scale_a), "r"(scale_b), "r"((unsigned)add) : "memory");
}
// CTAS 128 x n products of e4m3 codes; `byte` of its columns' words is the scale.
template <int CTAS>
__device__ __forceinline__ unsigned scaled_shape(unsigned n, unsigned byte) {
  return byte << 4 | (n >> 3) << 17 | 1u << 23 | (CTAS * 128u >> 4) << 24 | byte << 29;
}
// The mbarrier's phase counts this thread's products and copies so far as one
// arrival (CTAS 2: the barriers at this place in both CTAs).
template <int CTAS>
__device__ __forceinline__ void commit_to(unsigned bar) {
  if constexpr (CTAS == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar), "h"((unsigned short)3) : "memory");
}

}  // namespace tc
}  // namespace xp
