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
// One warp copies boxes of 128 columns into a ring of stages, one issues the
// products, two bring scales for four blocks at a time, and sixteen keep the
// tile's sums in registers: TMEM's are added to them after each 32 blocks, since
// the tensor core's own additions round towards zero and would be off by a few
// 2^-24 for each thousand columns.  While they are stored the next tile's products
// run.  Large products are made by pairs of CTAs, 256 rows of B at a time, half of
// A's rows in each's shared memory, which then has to deliver 256 bytes for what a
// CTA alone reads 384 for.  Where tiles are few, the CTAs of a cluster share one:
// each sums a part of the columns, and they add their sums up through shared
// memory, in the order of their ranks.  (A copy lands in the CTA that asks for it
// alone: no load here names several CTAs, so that operands may lie in any memory
// that the device reaches.)
//
// Every wait has a limit.  A warp that gives one up does its part no more: it
// arrives at no barrier again, so no other warp is told what is not so, and those
// that it keeps waiting give up in their turn.  Sums that were not read become NaN
// in C.  Before the CTA ends, its own copies and products have ended too, however
// far its warps and those of its pair have come.
#include <algorithm>

#include "xp_model_internal.h"
#include "xp_scales.h"
#include "xp_tcgen05.cuh"
#include "xp_train_device.cuh"

namespace xp {
namespace {

typedef unsigned long long u64;

constexpr int kScaleWarps = 2;                    // beside one that copies, one for the products
constexpr int kFirstStoreWarp = 2 + kScaleWarps;
constexpr int kStoreWarps = 16;
constexpr int kThreads = 32 * (kFirstStoreWarp + kStoreWarps);
constexpr int kRows = 128;                        // of B in a CTA's tile
constexpr unsigned kBoxCols = 128;                // a block's codes: 128 bytes
constexpr unsigned kRowsBytes = kRows * kBoxCols;
constexpr int kMaxStages = 12;
constexpr unsigned kScaleSlots = 4;               // of four blocks' scales each
constexpr unsigned kScaleBytes = 512 + 2 * 512;
constexpr unsigned kSharedBytes = 212 * 1024;     // stages and scales
constexpr unsigned kTmemColumns = 512;
constexpr unsigned kChunk = 32;                   // blocks between two readings of TMEM's sums
constexpr unsigned kMaxSplit = 8;
constexpr u64 kDrainNs = 2000000000ull;           // a limit for what is on its way when a wait was given up

static_assert(kScaleSlots == 2 * kScaleWarps, "a slot's phases are all waited for by the one warp that fills it");

__device__ unsigned stalled_warps;

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
                                            unsigned blocks, int lane) {
  const unsigned last = (rows - 1) >> shift;
  unsigned w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const unsigned row = row0 + lane + 32 * i;
    w[i] = row < rows ? scale_word(scales + (u64)(row >> shift) * pitch, group, blocks, row >> shift == last) : 0x7f7f7f7fu;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float4 load_remote(unsigned smem, unsigned rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(tc::in_cta(smem, rank)) : "memory");
  return v;
}

// The first n of N elements of C, `step` apart; what is there is read before anything is written.
template <int N>
__device__ __forceinline__ void put(const Matmul8Params& p, u64 at, u64 step, unsigned n, const float (&v)[N]) {
  if (p.out_bf16) {
    __nv_bfloat16* c = static_cast<__nv_bfloat16*>(p.c) + at;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < n) c[i * step] = __float2bfloat16_rn(v[i]);
    return;
  }
  float* c = static_cast<float*>(p.c) + at;
  float old[N];
#pragma unroll
  for (int i = 0; i < N; ++i) old[i] = p.accumulate && i < n ? c[i * step] : 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < n) c[i * step] = p.accumulate ? old[i] + v[i] : v[i];
}

// What a CTA, or a pair, still has on its way when a wait was given up and its
// warps are through; boxes: how many each CTA asked for.  (A function that calls
// none, as inlined, or with calls of its own, it cost the kernel registers: 8.6 us
// for one row of 4096 x 4096, 7.3 so.)
template <int CTAS>
__device__ __noinline__ void end_copies_and_products(Bars& bars, const unsigned* boxes, unsigned stages, unsigned stage_bytes) {
  const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (CTAS == 2 && tc::cluster_rank() != 0) return;   // the leader has the barriers
  if (warp == 0 && lane == 0) {
    // each stage's last box, which one CTA of a pair alone may have asked for
    const unsigned mine = boxes[0], other = boxes[CTAS - 1], n = max(mine, other);
    for (unsigned i = n >= stages ? n - stages : 0; i < n; ++i) {
      const unsigned bar = tc::smem_of(bars.full + i % stages);
      if (i >= other) tc::bar_uncount(bar, stage_bytes);
      if (i >= mine) tc::bar_expect(bar, stage_bytes);
      tc::bar_wait_here(bar, (i / stages) & 1, kDrainNs);
    }
  }
  if (warp == 1) {   // which issued the products
    if (tc::elected()) tc::commit_to<CTAS>(tc::smem_of(&bars.drained));
    tc::bar_wait_here(tc::smem_of(&bars.drained), 0, kDrainNs);
    tc::fence_before();
  }
  __syncwarp();
}

// CTAS: of a pair (2), or alone or in a cluster that shares a tile (1).
template <int CTAS>
__global__ void __launch_bounds__(kThreads, 1) matmul8_kernel(const __grid_constant__ Matmul8Params p) {
  extern __shared__ uint8_t raw[];
  __shared__ Bars bars;
  __shared__ unsigned tmem_at;
  __shared__ unsigned gave_up;          // a warp of this CTA, or of its pair
  __shared__ unsigned boxes[CTAS];      // that were asked for, by each CTA of a pair: in the leader's
  const unsigned base = (tc::smem_of(raw) + 1023u) & ~1023u;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const unsigned stages = p.stages, bn = p.bn, q_box = bn / CTAS, stage_bytes = kRowsBytes + q_box * kBoxCols;
  const unsigned scales_at = base + stages * stage_bytes;
  const unsigned full = tc::smem_of(bars.full), empty = tc::smem_of(bars.empty);
  const unsigned scales_full = tc::smem_of(bars.scales_full), scales_empty = tc::smem_of(bars.scales_empty);
  const unsigned sums_full = tc::smem_of(bars.sums_full), sums_empty = tc::smem_of(bars.sums_empty);
  const unsigned nsums = p.nsums, q_lines = (bn + 127) / 128, slot_columns = 4 + 4 * q_lines;
  const unsigned rank = CTAS == 2 || p.split > 1 ? tc::cluster_rank() : 0;
  const bool leader = CTAS == 1 || rank == 0;   // of a pair: it issues the products, and keeps the barriers they wait for

  if (warp == 0 && lane == 0) {
    tc::prefetch_map(&p.p_map);
    tc::prefetch_map(&p.q_map);
  }
  if (warp == 1 && lane == 0) {
    gave_up = 0;
    for (unsigned i = 0; i < stages; ++i) {
      tc::bar_init(full + 8 * i, 1);
      tc::bar_init(empty + 8 * i, 1);
    }
    tc::bar_init(tc::smem_of(&bars.drained), 1);
    for (unsigned i = 0; i < kScaleSlots; ++i) {
      tc::bar_init(scales_full + 8 * i, CTAS);
      tc::bar_init(scales_empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::bar_init(sums_full + 8 * i, 1);
      tc::bar_init(sums_empty + 8 * i, CTAS * kStoreWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 2) tc::tmem_alloc<CTAS>(tc::smem_of(&tmem_at), kTmemColumns);
  tc::fence_before();
  __syncthreads();
  if (CTAS == 2) tc::cluster_meet();
  tc::fence_after();
  const unsigned tmem = __shfl_sync(0xffffffffu, tmem_at, 0);   // the same for the warp, as the compiler then knows
  wait_for_predecessors();
  let_successor_start();

  const unsigned sharers = CTAS * p.split;   // CTAs of a tile
  const unsigned first_tile = blockIdx.x / sharers, tile_step = gridDim.x / sharers, ntiles = p.tiles_p * p.tiles_q;
  const unsigned part = CTAS == 2 ? 0 : rank;
  const unsigned k0 = (unsigned)((u64)p.kblocks * part / p.split), k1 = (unsigned)((u64)p.kblocks * (part + 1) / p.split);
  constexpr unsigned kTileRows = CTAS * kRows;
  const unsigned p_first = CTAS == 2 ? rank * kRows : 0, q_first = CTAS == 2 ? rank * q_box : 0;   // of the tile's rows, in this CTA
  bool ok = true;

  if (warp == 0) {
    const unsigned full_at = CTAS == 2 ? tc::in_cta(full, 0) : full;
    unsigned n = 0, s = 0, turn = 0;   // boxes brought so far; the stage of the next, and how often the ring went round
    for (unsigned t = first_tile; t < ntiles && ok; t += tile_step) {
      unsigned tp, tq;
      tile_at(p, t, tp, tq);
      const int row_p = tp * kTileRows + p_first, row_q = tq * bn + q_first;
      for (unsigned kb = k0; kb < k1; ++kb, ++n) {
        if (turn > 0 && !(ok = __all_sync(0xffffffffu, tc::bar_wait(empty + 8 * s, (turn - 1) & 1, p.limit_ns)))) break;
        if (tc::elected()) {
          const unsigned at = base + s * stage_bytes;
          if (leader) tc::bar_expect(full + 8 * s, CTAS * stage_bytes);
          tc::load_box<CTAS>(at, &p.p_map, kb * kBoxCols, row_p, full_at + 8 * s);
          tc::load_box<CTAS>(at + kRowsBytes, &p.q_map, kb * kBoxCols, row_q, full_at + 8 * s);
        }
        if (++s == stages) s = 0, ++turn;
      }
    }
    if (lane == 0) {
      if constexpr (CTAS == 2)
        tc::store_in_cta(tc::smem_of(boxes + rank), 0, n);
      else
        boxes[0] = n;
    }
  } else if (warp == 1) {
    if (leader) {
      unsigned s = 0, phase = 0, slot = 0, slot_phase = 0, sums = 0, turn = 0;
      for (unsigned t = first_tile; t < ntiles && ok; t += tile_step) {
        for (unsigned from = k0; from < k1 && ok; from += kChunk) {
          const unsigned d = tmem + sums * bn, to = min(from + kChunk, k1);
          if (turn > 0 && !(ok = __all_sync(0xffffffffu, tc::bar_wait(sums_empty + 8 * sums, (turn - 1) & 1, p.limit_ns)))) break;
          for (unsigned kb = from; kb < to; ++kb) {
            const unsigned at = base + s * stage_bytes, scale_p = tmem + nsums * bn + slot * slot_columns, scale_q = scale_p + 4;
            const bool more = kb == k0 || kb % 4 == 0, last = kb + 1 == k1 || kb % 4 == 3;
            ok = tc::bar_wait(full + 8 * s, phase, p.limit_ns) && (!more || tc::bar_wait<CTAS == 2>(scales_full + 8 * slot, slot_phase, p.limit_ns));
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            tc::fence_after();
            if (tc::elected()) {
              if (more) {   // the next four blocks' scales
                const unsigned in = scales_at + slot * kScaleBytes;
                tc::copy_scales<CTAS>(scale_p, tc::rows16(in));
                tc::copy_scales<CTAS>(scale_q, tc::rows16(in + 512));
                if (q_lines > 1) tc::copy_scales<CTAS>(scale_q + 4, tc::rows16(in + 1024));
              }
              const unsigned shape = tc::scaled_shape<CTAS>(bn, kb % 4);
              const u64 a = tc::rows128(at), b = tc::rows128(at + kRowsBytes);
#pragma unroll
              for (int i = 0; i < 4; ++i) tc::mma_scaled<CTAS>(d, a + 2 * i, b + 2 * i, shape, scale_p, scale_q, kb != from || i > 0);
              tc::commit_to<CTAS>(empty + 8 * s);
              // a slot is free, here and in TMEM, when the last products that read it are done
              if (last) tc::commit_to<CTAS>(scales_empty + 8 * slot);
              if (kb + 1 == to) tc::commit_to<CTAS>(sums_full + 8 * sums);
            }
            __syncwarp();
            if (last && ++slot == kScaleSlots) slot = 0, slot_phase ^= 1;
            if (++s == stages) s = 0, phase ^= 1;
          }
          if (++sums == nsums) sums = 0, ++turn;
        }
      }
    }
  } else if (warp < kFirstStoreWarp) {
    // A warp brings two groups of four blocks' scales at a time: the fence between its loads and the tensor core's
    // copies waits for all that the warp has on its way, and one group after another takes 2800 cycles each, longer
    // than four blocks' products (8192 x 16384 x 4096: 364 us with one such warp, 335 with four groups on their way).
    const unsigned scales_full_at = CTAS == 2 ? tc::in_cta(scales_full, 0) : scales_full;
    const unsigned g0 = k0 / 4, per_tile = k0 < k1 ? (k1 + 3) / 4 - g0 : 0;
    const unsigned mine = first_tile < ntiles ? (ntiles - first_tile + tile_step - 1) / tile_step * per_tile : 0;
    unsigned at = 2 * (warp - 2), tile = first_tile;   // the group within its tile
    for (unsigned n = 2 * (warp - 2); n < mine && ok; n += 2 * kScaleWarps) {
      uint4 line[2][3];
#pragma unroll
      for (unsigned u = 0; u < 2; ++u, ++at) {
        while (at >= per_tile) at -= per_tile, tile += tile_step;
        if (n + u >= mine) break;
        unsigned tp, tq;
        tile_at(p, tile, tp, tq);
        line[u][0] = scale_line(p.p_scales, p.p_pitch, p.p_shift, tp * kTileRows + p_first, p.p_rows, g0 + at, p.kblocks, lane);
        line[u][1] = scale_line(p.q_scales, p.q_pitch, p.q_shift, tq * bn, p.q_rows, g0 + at, p.kblocks, lane);
        if (q_lines > 1) line[u][2] = scale_line(p.q_scales, p.q_pitch, p.q_shift, tq * bn + 128, p.q_rows, g0 + at, p.kblocks, lane);
      }
      at += 2 * (kScaleWarps - 1);
#pragma unroll
      for (unsigned u = 0; u < 2; ++u) {
        const unsigned slot = (n + u) % kScaleSlots, to = scales_at + slot * kScaleBytes + 16 * lane;
        if (n + u >= mine) break;
        if (n + u >= kScaleSlots && !(ok = __all_sync(0xffffffffu, tc::bar_wait(scales_empty + 8 * slot, ((n + u) / kScaleSlots - 1) & 1, p.limit_ns)))) break;
#pragma unroll
        for (unsigned i = 0; i < 3; ++i)
          if (i <= q_lines)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(to + 512 * i), "r"(line[u][i].x), "r"(line[u][i].y), "r"(line[u][i].z), "r"(line[u][i].w) : "memory");
      }
      if (!ok) break;
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane < 2 && n + lane < mine) tc::bar_arrive_cluster(scales_full_at + 8 * ((n + lane) % kScaleSlots));
    }
  } else {
    // a warp has 32 rows of B, and every fourth 16 of A's
    const unsigned quarter = warp & 3, first = 16 * ((warp - kFirstStoreWarp) >> 2), row = 32 * quarter + lane;
    const unsigned sums_empty_at = CTAS == 2 ? tc::in_cta(sums_empty, 0) : sums_empty;
    unsigned sums = 0, phase = 0;
    for (unsigned t = first_tile; t < ntiles; t += tile_step) {
      float v[4][16];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 16; ++i) v[j][i] = 0.f;
      for (unsigned from = k0; from < k1; from += kChunk) {
        if (!ok || !(ok = __all_sync(0xffffffffu, tc::bar_wait(sums_full + 8 * sums, phase, p.limit_ns)))) break;
        tc::fence_after();
        // (columns past bn are read too, within TMEM's 512, and not used)
        const unsigned at = tmem + sums * bn + first + ((32 * quarter) << 16);
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
          if (64 * j + first >= bn) break;
          float f[2][16];
          tc::tmem_load16(at + 64 * j, f[0]);
          tc::tmem_load16(at + 64 * j + 64, f[1]);
          tc::tmem_wait();
          tc::landed(f[0]);
          tc::landed(f[1]);
#pragma unroll
          for (int i = 0; i < 16; ++i) v[j][i] += f[0][i], v[j + 1][i] += f[1][i];
        }
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::bar_arrive_relaxed(sums_empty_at + 8 * sums);
        if (++sums == nsums) sums = 0, phase ^= 1;
      }
      if (!ok) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int i = 0; i < 16; ++i) v[j][i] = __int_as_float(0x7fffffff);
      }
      unsigned tp, tq;
      tile_at(p, t, tp, tq);
      const unsigned n = tp * kTileRows + p_first + row, m0 = tq * bn;
      const unsigned there = n < p.p_rows ? min(bn, p.q_rows - m0) : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const unsigned c = 64 * j + first;
        if (p.split == 1) {
          if (c < there) put<16>(p, (u64)(m0 + c) * p.c_stride + n, p.c_stride, there - c, v[j]);
        } else if (c < bn && ok) {   // (else boxes may still land there)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(base + ((c + i) * kRows + row) * 4), "f"(v[j][i]) : "memory");
        }
      }
    }
  }
  if (!ok && lane == 0) {
    atomicAdd(&stalled_warps, 1u);
    gave_up = 1;
    if constexpr (CTAS == 2) tc::store_in_cta(tc::smem_of(&gave_up), rank ^ 1, 1);
  }
  __syncwarp();
  if (CTAS == 1 && p.split > 1) {
    tc::cluster_meet();
    unsigned tp, tq;
    tile_at(p, first_tile, tp, tq);
    // a thread adds up four of the 128 rows of B at one of A's, which go to the CTAs in turn
    const unsigned row = 4 * lane, n = tp * kRows + row;
    const unsigned missing = lane < p.split ? tc::load_in_cta(tc::smem_of(&gave_up), lane) : 0;
    for (unsigned j = rank + p.split * warp; j < bn && tq * bn + j < p.q_rows; j += p.split * (kThreads / 32)) {
      float4 part[kMaxSplit];
#pragma unroll
      for (unsigned r = 0; r < kMaxSplit; ++r)
        if (r < p.split) part[r] = load_remote(base + (j * kRows + row) * 4, r);
      float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (unsigned r = 0; r < kMaxSplit; ++r)
        if (r < p.split) v[0] += part[r].x, v[1] += part[r].y, v[2] += part[r].z, v[3] += part[r].w;
      if (__any_sync(0xffffffffu, missing)) v[0] = v[1] = v[2] = v[3] = __int_as_float(0x7fffffff);
      if (n < p.p_rows) put<4>(p, (u64)(tq * bn + j) * p.c_stride + n, 1, p.p_rows - n, v);
    }
  }
  tc::fence_before();
  if (CTAS == 2 || p.split > 1)
    tc::cluster_meet();   // nobody reads or signals this CTA's shared memory any more
  else
    __syncthreads();
  if (gave_up) {   // in both CTAs of a pair
    end_copies_and_products<CTAS>(bars, boxes, p.stages, kRowsBytes + p.bn / CTAS * kBoxCols);
    if (CTAS == 2)
      tc::cluster_meet();
    else
      __syncthreads();
  }
  if (warp == 2) {
    tc::fence_after();
    tc::tmem_free<CTAS>(tmem, kTmemColumns);
  }
}

// Pairs of CTAs that fit on the device at a time.
int pair_count(int sms) {
  static PerDevice known;
  return known.get([sms](int) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSharedBytes;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int n = 0;
    if (allow_dynamic_smem(matmul8_kernel<2>) != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, matmul8_kernel<2>, &cfg) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      n = std::max(1, sms / 2);
    }
    return n;
  });
}

}  // namespace

cudaError_t launch_matmul8(Matmul8Params& p, int sms, cudaStream_t st) {
  const unsigned stage = kRowsBytes + p.bn / p.ctas * kBoxCols;
  p.stages = (kSharedBytes - 1024 - kScaleSlots * kScaleBytes) / stage;
  if (p.stages > (unsigned)kMaxStages) p.stages = kMaxStages;
  // two chunks' sums at a time where they fit beside the scales
  const unsigned slot = 4 + 4 * ((p.bn + 127) / 128);
  p.nsums = 2 * p.bn + kScaleSlots * slot <= kTmemColumns ? 2 : 1;
  const unsigned tiles = p.tiles_p * p.tiles_q;
  // (a CTA has its SM to itself, so clusters do not hold up the kernel that drains before them: 310 us with programmatic
  // dependence and 324 without at 8192 x 16384 x 4096, 8.7 and 9.6 for one row of 4096 x 4096)
  if (p.ctas == 2)
    return launch_clusters(matmul8_kernel<2>, dim3(2 * std::min(tiles, (unsigned)pair_count(sms))), kThreads, kSharedBytes, 2, true, st, p);
  const unsigned grid = p.split > 1 ? tiles * p.split : tiles < (unsigned)sms ? tiles : (unsigned)sms;
  return launch_clusters(matmul8_kernel<1>, dim3(grid), kThreads, kSharedBytes, (int)p.split, true, st, p);
}

// (The copy by itself waits for the legacy default stream and those that wait for it, not for streams that do not.)
cudaError_t matmul8_stalls(unsigned* n) {
  const cudaError_t e = cudaDeviceSynchronize();
  return e != cudaSuccess ? e : cudaMemcpyFromSymbol(n, stalled_warps, sizeof *n);
}

}  // namespace xp
