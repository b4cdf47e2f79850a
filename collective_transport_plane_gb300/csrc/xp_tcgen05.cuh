// The fifth-generation tensor core's instructions, its memory (TMEM) and the
// tiled copies that feed it, as the product of 8-bit matrices uses them.
#pragma once

#include <cuda.h>

#include <cstdint>

namespace xp {
namespace tc {

__device__ __forceinline__ unsigned smem_of(const void* p) { return (unsigned)__cvta_generic_to_shared(p); }

// ---- mbarriers, all waits with a limit
__device__ __forceinline__ void bar_init(unsigned bar, unsigned count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(unsigned bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(unsigned bar, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(unsigned bar, unsigned parity) {
  unsigned ok;
  asm volatile("{\n.reg .pred p;\nmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\nselp.u32 %0, 1, 0, p;\n}"
               : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// A wait gives up after two seconds of the GPU's clock (no wait here is for
// another kernel, and the longest loop of products takes milliseconds).
constexpr unsigned long long kLimitNs = 2000000000ull;
__device__ __forceinline__ unsigned long long clock_ns() {
  unsigned long long t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
__device__ __noinline__ bool bar_wait_long(unsigned bar, unsigned parity) {
  const unsigned long long start = clock_ns();
  do {
    for (int i = 0; i < 64; ++i)
      if (bar_try(bar, parity)) return true;
  } while (clock_ns() - start < kLimitNs);
  return false;
}
__device__ __forceinline__ bool bar_wait(unsigned bar, unsigned parity) { return bar_try(bar, parity) || bar_wait_long(bar, parity); }

// ---- tiled copies into shared memory
__device__ __forceinline__ void prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
// the box of `m` whose first element is column x of row y
__device__ __forceinline__ void load_box(unsigned smem, const CUtensorMap* m, int x, int y, unsigned bar) {
  asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
               ::"r"(smem), "l"(m), "r"(x), "r"(y), "r"(bar) : "memory");
}

// ---- TMEM: 128 lanes of 512 columns of 32 bits; an address is lane << 16 | column
__device__ __forceinline__ void tmem_alloc(unsigned result_smem, unsigned columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(result_smem), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(unsigned at, unsigned columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}
// 16 columns of the warp's 32 lanes, a lane's into its own registers
__device__ __forceinline__ void tmem_load16(unsigned at, float (&v)[16]) {
  unsigned u[16];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]), "=r"(u[8]), "=r"(u[9]),
                 "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15])
               : "r"(at) : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(u[i]);
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
// 32 rows of 16 bytes to 4 columns, the same for each 32 lanes.
__device__ __forceinline__ void copy_scales(unsigned tmem, unsigned long long rows) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(rows) : "memory");
}
// d = [d +] a b^T over 32 columns of codes (e4m3), each row's 32 columns times
// the power of two that its scale byte says.
__device__ __forceinline__ void mma_scaled(unsigned d, unsigned long long a, unsigned long long b, unsigned shape, unsigned scale_a,
                                           unsigned scale_b, bool add) {
  asm volatile("{\n.reg .pred p;\nsetp.ne.u32 p, %6, 0;\n"
               "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}"
               ::"r"(d), "l"(a), "l"(b), "r"(shape), "r"(scale_a), "r"(scale_b), "r"((unsigned)add) : "memory");
}
// 128 x n products of e4m3 codes; `byte` of its columns' words is the scale.
__device__ __forceinline__ unsigned scaled_shape(unsigned n, unsigned byte) {
  return byte << 4 | (n >> 3) << 17 | 1u << 23 | (128u >> 4) << 24 | byte << 29;
}
// The mbarrier's phase counts this thread's products and copies so far as one arrival.
__device__ __forceinline__ void commit_to(unsigned bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

}  // namespace tc
}  // namespace xp
