// The product of two matrices of 8-bit codes with a scale for each block of
// 128 columns, C = A B^T (include/xp_model.h), on the tensor cores.
//
// A scale is a power of two, so the tensor core applies it: a product over 32
// columns takes each row's scale byte from TMEM, and sums stay in fp32 there
// from the first column to the last.  B's rows (the output's columns) are the
// product's 128 rows and A's rows its columns: a lane of TMEM is then a column
// of C, and a warp stores 32 neighbouring elements of it, at any alignment.
// Few rows of A take few columns, and the same kernel reads a weight at the
// memory's rate for one token.
//
// A CTA works on tiles of 128 x `bn`, one after another: one thread copies
// boxes of 128 columns into a ring of stages, one issues the products, a warp
// brings scales for four blocks at a time, and four warps store the last tile's
// sums while the next one's are made.  Where tiles are few, the CTAs of a
// cluster share one: each sums a part of the columns, and they add their sums up
// through shared memory, in the order of their ranks.
#include "xp_model_internal.h"
#include "xp_tcgen05.cuh"
#include "xp_train_device.cuh"

namespace xp {
namespace {

typedef unsigned long long u64;

constexpr int kThreads = 256;
constexpr int kRows = 128;                        // of B in a tile
constexpr unsigned kBoxCols = 128;                // a block's codes: 128 bytes
constexpr unsigned kRowsBytes = kRows * kBoxCols;
constexpr int kMaxStages = 12;
constexpr unsigned kScaleSlots = 4;               // of four blocks' scales each, at most
constexpr unsigned kScaleBytes = 512 + 2 * 512;
constexpr unsigned kSharedBytes = 212 * 1024;     // stages and scales
constexpr unsigned kTmemColumns = 512;

__device__ unsigned stalled_ctas;

struct Bars {
  u64 full[kMaxStages], empty[kMaxStages];
  u64 scales_full[kScaleSlots], scales_empty[kScaleSlots];
  u64 sums_full[2], sums_empty[2];
  u64 drained;
};

// Which tile is the t-th: 16 tiles down B's rows before the next of A's, so
// that what runs at a time shares both operands in L2.
__device__ __forceinline__ void tile_at(const Matmul8Params& p, unsigned t, unsigned& tp, unsigned& tq) {
  const unsigned per = 16 * p.tiles_q, group = t / per, first = group * 16, in = t - group * per;
  const unsigned high = min(16u, p.tiles_p - first);
  tp = first + in % high;
  tq = in / high;
}

// The words of four blocks' scales that lane l's line holds, of the 128 rows
// from row0: rows l, l + 32, l + 64 and l + 96.  Rows that are not there get 2^0.
__device__ __forceinline__ uint4 scale_line(const uint8_t* scales, u64 pitch, int shift, unsigned row0, unsigned rows, unsigned group,
                                            int lane) {
  unsigned w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned row = row0 + lane + 32 * i;
    w[i] = row < rows ? *reinterpret_cast<const unsigned*>(scales + (u64)(row >> shift) * pitch + 4ull * group) : 0x7f7f7f7fu;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ float load_remote(unsigned smem, unsigned rank) {
  unsigned r;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
  return v;
}

// The first n of N elements of C, a row apart from the next; what is there is read before anything is written.
template <int N>
__device__ __forceinline__ void put(const Matmul8Params& p, u64 at, unsigned n, const float (&v)[N]) {
  if (p.out_bf16) {
    __nv_bfloat16* c = static_cast<__nv_bfloat16*>(p.c) + at;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) c[i * p.c_stride] = __float2bfloat16_rn(v[i]);
    return;
  }
  float* c = static_cast<float*>(p.c) + at;
  float old[N];
#pragma unroll
  for (int i = 0; i < N; ++i) old[i] = p.accumulate && i < n ? c[i * p.c_stride] : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < n) c[i * p.c_stride] = p.accumulate ? old[i] + v[i] : v[i];
}

__global__ void __launch_bounds__(kThreads, 1) matmul8_kernel(const __grid_constant__ Matmul8Params p) {
  extern __shared__ uint8_t raw[];
  __shared__ Bars bars;
  __shared__ unsigned tmem_at;
  const unsigned base = (tc::smem_of(raw) + 1023u) & ~1023u;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned stages = p.stages, bn = p.bn, stage_bytes = kRowsBytes + bn * kBoxCols;
  const unsigned scales_at = base + stages * stage_bytes;
  const unsigned full = tc::smem_of(bars.full), empty = tc::smem_of(bars.empty);
  const unsigned scales_full = tc::smem_of(bars.scales_full), scales_empty = tc::smem_of(bars.scales_empty);
  const unsigned sums_full = tc::smem_of(bars.sums_full), sums_empty = tc::smem_of(bars.sums_empty);
  const unsigned drained = tc::smem_of(&bars.drained);
  const unsigned nsums = p.nsums, nslots = p.slots, q_lines = (bn + 127) / 128, slot_columns = 4 + 4 * q_lines;

  if (warp == 0 && lane == 0) {
    tc::prefetch_map(&p.p_map);
    tc::prefetch_map(&p.q_map);
  }
  if (warp == 1 && lane == 0) {
    for (unsigned i = 0; i < stages; ++i) {
      tc::bar_init(full + 8 * i, 1);
      tc::bar_init(empty + 8 * i, 1);
    }
    tc::bar_init(drained, 1);
    for (unsigned i = 0; i < kScaleSlots; ++i) {
      tc::bar_init(scales_full + 8 * i, 1);
      tc::bar_init(scales_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::bar_init(sums_full + 8 * i, 1);
      tc::bar_init(sums_empty + 8 * i, 4);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) tc::tmem_alloc(tc::smem_of(&tmem_at), kTmemColumns);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const unsigned tmem = tmem_at;
  wait_for_predecessors();
  let_successor_start();

  const unsigned rank = p.split > 1 ? cluster_rank() : 0;
  const unsigned first_tile = blockIdx.x / p.split, tile_step = gridDim.x / p.split, ntiles = p.tiles_p * p.tiles_q;
  const unsigned k0 = (unsigned)((u64)p.kblocks * rank / p.split), k1 = (unsigned)((u64)p.kblocks * (rank + 1) / p.split);
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      unsigned n = 0;   // boxes brought so far
      for (unsigned t = first_tile; t < ntiles && ok; t += tile_step) {
        unsigned tp, tq;
        tile_at(p, t, tp, tq);
        for (unsigned kb = k0; kb < k1; ++kb, ++n) {
          const unsigned s = n % stages, at = base + s * stage_bytes;
          if (n >= stages && !(ok = tc::bar_wait(empty + 8 * s, (n / stages - 1) & 1))) break;
          tc::bar_expect(full + 8 * s, stage_bytes);
          tc::load_box(at, &p.p_map, kb * kBoxCols, tp * kRows, full + 8 * s);
          tc::load_box(at + kRowsBytes, &p.q_map, kb * kBoxCols, tq * bn, full + 8 * s);
        }
      }
      if (!ok)   // what is in flight lands before the CTA goes
        for (unsigned i = n >= stages ? n - stages : 0; i < n; ++i) tc::bar_wait(full + 8 * (i % stages), (i / stages) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      unsigned n = 0, groups = 0, tiles = 0;
      for (unsigned t = first_tile; t < ntiles && ok; t += tile_step, ++tiles) {
        const unsigned sums = tiles % nsums, turn = tiles / nsums, d = tmem + sums * bn;
        if (turn > 0 && !(ok = tc::bar_wait(sums_empty + 8 * sums, (turn - 1) & 1))) break;
        tc::fence_after();
        unsigned slot = 0, scale_p = 0, scale_q = 0;
        for (unsigned kb = k0; kb < k1; ++kb, ++n) {
          const unsigned s = n % stages, at = base + s * stage_bytes;
          if (!(ok = tc::bar_wait(full + 8 * s, (n / stages) & 1))) break;
          if (kb == k0 || kb % 4 == 0) {   // the next four blocks' scales
            slot = groups % nslots;
            const unsigned from = scales_at + slot * kScaleBytes;
            if (!(ok = tc::bar_wait(scales_full + 8 * slot, (groups / nslots) & 1))) break;
            scale_p = tmem + nsums * bn + slot * slot_columns;
            scale_q = scale_p + 4;
            tc::fence_after();
            tc::copy_scales(scale_p, tc::rows16(from));
            for (unsigned i = 0; i < q_lines; ++i) tc::copy_scales(scale_q + 4 * i, tc::rows16(from + 512 + 512 * i));
            ++groups;
          }
          tc::fence_after();
          const unsigned shape = tc::scaled_shape(bn, kb % 4);
          const u64 a = tc::rows128(at), b = tc::rows128(at + kRowsBytes);
#pragma unroll
          for (int i = 0; i < 4; ++i) tc::mma_scaled(d, a + 2 * i, b + 2 * i, shape, scale_p, scale_q, kb != k0 || i > 0);
          tc::commit_to(empty + 8 * s);
          // a slot is free, here and in TMEM, when the last products that read it are done
          if (kb + 1 == k1 || kb % 4 == 3) tc::commit_to(scales_empty + 8 * slot);
        }
        if (ok) tc::commit_to(sums_full + 8 * sums);
      }
      if (!ok) {   // what was issued ends before TMEM is given back
        tc::commit_to(drained);
        tc::bar_wait(drained, 0);
      }
    }
  } else if (warp == 2) {
    unsigned n = 0;
    for (unsigned t = first_tile; t < ntiles && ok; t += tile_step) {
      unsigned tp, tq;
      tile_at(p, t, tp, tq);
      for (unsigned g = k0 / 4; g * 4 < k1 && k0 < k1; ++g, ++n) {
        const unsigned slot = n % nslots, to = scales_at + slot * kScaleBytes + 16 * lane;
        uint4 line[3];
        line[0] = scale_line(p.p_scales, p.p_pitch, p.p_shift, tp * kRows, p.p_rows, g, lane);
#pragma unroll
        for (unsigned i = 0; i < 2; ++i)
          if (i < q_lines) line[1 + i] = scale_line(p.q_scales, p.q_pitch, p.q_shift, tq * bn + 128 * i, p.q_rows, g, lane);
        if (n >= nslots && !(ok = __all_sync(0xffffffffu, tc::bar_wait(scales_empty + 8 * slot, (n / nslots - 1) & 1)))) break;
#pragma unroll
        for (unsigned i = 0; i < 3; ++i)
          if (i <= q_lines)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + 512 * i), "r"(line[i].x), "r"(line[i].y), "r"(line[i].z), "r"(line[i].w) : "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) tc::bar_arrive(scales_full + 8 * slot);
      }
    }
  } else if (warp >= 4) {
    const unsigned row = 32 * (warp - 4) + lane;
    unsigned tiles = 0;
    for (unsigned t = first_tile; t < ntiles; t += tile_step, ++tiles) {
      unsigned tp, tq;
      tile_at(p, t, tp, tq);
      const unsigned sums = tiles % nsums, turn = tiles / nsums, n = tp * kRows + row, m0 = tq * bn;
      const bool none = k0 == k1;
      ok = ok && (none || __all_sync(0xffffffffu, tc::bar_wait(sums_full + 8 * sums, turn & 1)));
      tc::fence_after();
      const unsigned there = n < p.p_rows ? p.q_rows - m0 : 0;
      for (unsigned j = 0; j < bn; j += 16) {
        float v[16];
        if (ok && !none) {
          tc::tmem_load16(tmem + sums * bn + j + ((32u * (warp - 4)) << 16), v);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = none ? 0.f : __int_as_float(0x7fffffff);
        }
        if (p.split == 1) {
          put<16>(p, (u64)(m0 + j) * p.c_stride + n, j < there ? there - j : 0, v);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + ((j + i) * kRows + row) * 4), "f"(v[i]) : "memory");
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(sums_empty + 8 * sums);
    }
  }
  if (!ok && lane == 0) atomicAdd(&stalled_ctas, 1u);
  __syncwarp();
  if (p.split > 1) {
    cluster_meet();
    unsigned tp, tq;
    tile_at(p, first_tile, tp, tq);
    const unsigned row = threadIdx.x % kRows, n = tp * kRows + row;
    for (unsigned j = rank + p.split * (threadIdx.x / kRows); j < bn && tq * bn + j < p.q_rows; j += p.split * (kThreads / kRows)) {
      float v[1] = {0.f};
      for (unsigned r = 0; r < p.split; ++r) v[0] += load_remote(base + (j * kRows + row) * 4, r);
      put<1>(p, (u64)(tq * bn + j) * p.c_stride + n, n < p.p_rows, v);
    }
    cluster_meet();
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 2) {
    tc::fence_after();
    tc::tmem_free(tmem, kTmemColumns);
  }
}

}  // namespace

cudaError_t launch_matmul8(Matmul8Params& p, int sms, cudaStream_t st) {
  const unsigned stage = kRowsBytes + p.bn * kBoxCols;
  p.stages = (kSharedBytes - 1024 - kScaleSlots * kScaleBytes) / stage;
  if (p.stages > (unsigned)kMaxStages) p.stages = kMaxStages;
  // two tiles' sums at a time where they fit beside two slots of scales
  const unsigned slot = 4 + 4 * ((p.bn + 127) / 128);
  p.nsums = 2 * (p.bn + slot) <= kTmemColumns ? 2 : 1;
  p.slots = p.nsums * p.bn + kScaleSlots * slot <= kTmemColumns ? kScaleSlots : 2;
  const unsigned tiles = p.tiles_p * p.tiles_q;
  const unsigned grid = p.split > 1 ? tiles * p.split : tiles < (unsigned)sms ? tiles : (unsigned)sms;
  return launch_dependent(matmul8_kernel, dim3(grid), kThreads, kSharedBytes, (int)p.split, st, p);
}

cudaError_t matmul8_stalls(unsigned* n) { return cudaMemcpyFromSymbol(n, stalled_ctas, sizeof *n); }

}  // namespace xp
