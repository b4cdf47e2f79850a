// The root-mean-square norm with the residual's addition and an output in 8
// bits, and its backward pass (include/xp_model.h).
//
// Both directions read and write every element once and compute little on it:
// HBM bounds them.  A row's threads keep it in registers between its sum and
// its outputs, or in shared memory, backward (rows of more than 16384 columns,
// 8192 of fp32 or of unaligned rows, are read twice).  Blocks of 128 columns lie
// in one warp's units, so a block's scale is a maximum over lanes.
#include <algorithm>

#include "xp_code8.cuh"
#include "xp_model_internal.h"
#include "xp_train_device.cuh"

namespace xp {
namespace {

typedef __nv_bfloat16 bf16;
typedef unsigned long long u64;

// ---- units: what a thread takes at a time.  WIDE: 16 bytes side by side.  In
// rows that do not allow it (lengths, strides or addresses that are no multiple
// of 16 bytes) a warp's lanes take neighbouring elements, 128 columns at a time.
template <typename T, bool WIDE>
constexpr int kUnit = WIDE ? 16 / (int)sizeof(T) : 4;

// A row's thread, of `threads`: the first column of its unit k, and what its
// unit's elements are apart.
template <typename T, bool WIDE>
__device__ __forceinline__ unsigned column(unsigned tid, unsigned threads, unsigned k) {
  if constexpr (WIDE) return (tid + k * threads) * kUnit<T, WIDE>;
  return ((tid >> 5) + k * (threads >> 5)) * 128 + (tid & 31);
}
template <bool WIDE>
constexpr unsigned kApart = WIDE ? 1 : 32;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float v, float& x) { x = v; }
__device__ __forceinline__ void from_f(float v, bf16& x) { x = __float2bfloat16_rn(v); }
template <typename T>
__device__ __forceinline__ float rounded(float v) {
  T x;
  from_f(v, x);
  return to_f(x);
}

__device__ __forceinline__ unsigned pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const unsigned*>(&h);
}

// A unit whose first column is c, of a row of `cols`; zeros past its end.
template <typename T, bool WIDE, int V>
__device__ __forceinline__ void load(const T* row, unsigned c, unsigned cols, float (&f)[V]) {
  if constexpr (WIDE) {
    const uint4 q = c < cols ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0, 0, 0, 0);
    const unsigned w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        f[i] = __uint_as_float(w[i]);
      } else {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  } else {
    const T* at = row + c;
    const int n = (int)cols - (int)c;
    if (n > 32 * (V - 1)) {
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = to_f(at[32 * i]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) f[i] = 32 * i < n ? to_f(at[32 * i]) : 0.f;
    }
  }
}
template <typename T, bool WIDE, int V>
__device__ __forceinline__ void store(T* row, unsigned c, unsigned cols, const float (&f)[V]) {
  if constexpr (WIDE) {
    if (c >= cols) return;
    if constexpr (sizeof(T) == 4)
      *reinterpret_cast<float4*>(row + c) = make_float4(f[0], f[1], f[2], f[3]);
    else
      *reinterpret_cast<uint4*>(row + c) = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
  } else {
    T* at = row + c;
    const int n = (int)cols - (int)c;
    if (n > 32 * (V - 1)) {
#pragma unroll
      for (int i = 0; i < V; ++i) from_f(f[i], at[32 * i]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (32 * i < n) from_f(f[i], at[32 * i]);
    }
  }
}
// gamma's unit; ones where there is none (fp32 or bf16, its own alignment in `g`)
template <bool WIDE, int V>
__device__ __forceinline__ void load_gamma(const void* gamma, bool is_bf16, unsigned c, unsigned cols, float (&f)[V]) {
  if (!gamma) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = 1.f;
  } else if constexpr (!WIDE) {
    if (is_bf16)
      load<bf16, false>(static_cast<const bf16*>(gamma), c, cols, f);
    else
      load<float, false>(static_cast<const float*>(gamma), c, cols, f);
  } else if (c >= cols) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = 0.f;
  } else if (is_bf16) {
    const bf16* g = static_cast<const bf16*>(gamma) + c;
    const uint2 a = *reinterpret_cast<const uint2*>(g);
    const uint2 b = V == 8 ? *reinterpret_cast<const uint2*>(g + V - 4) : a;
    const unsigned w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    const float4* g = reinterpret_cast<const float4*>(static_cast<const float*>(gamma) + c);
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const float4 q = g[i];
      f[4 * i] = q.x, f[4 * i + 1] = q.y, f[4 * i + 2] = q.z, f[4 * i + 3] = q.w;
    }
  }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// The sum over a row's threads (whole warps), the same in each; every thread of
// the CTA calls it.  words: one per warp, two buffers in turn where it is
// called more than once.
__device__ __forceinline__ float row_sum(float v, float* words, unsigned threads) {
  v = warp_sum(v);
  if (threads == 32) return v;
  const unsigned warp = threadIdx.x >> 5, n = threads >> 5, first = warp / n * n;
  if ((threadIdx.x & 31) == 0) words[warp] = v;
  __syncthreads();
  v = 0.f;
  for (unsigned i = 0; i < n; ++i) v += words[first + i];
  return v;
}

// A unit's codes, and its block's scale by the lane that has its first columns.
template <typename T, bool WIDE, int V>
__device__ __forceinline__ void store8(const RmsForwardParams& p, u64 row, bool there, unsigned c, const float (&y)[V]) {
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < V; ++i) top = max(top, abs_bits(y[i]));
  constexpr int kBlockLanes = WIDE ? 128 / V : 32;
#pragma unroll
  for (int o = kBlockLanes / 2; o > 0; o /= 2) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (!there || c >= p.cols) return;
  const unsigned e = scale_of(top);
  const float inverse = inverse_of(e);
  if ((threadIdx.x & (kBlockLanes - 1)) == 0) p.y8_scales[row * p.y8_scales_stride + c / 128] = (uint8_t)e;
  uint8_t* out = p.y8 + row * p.y8_stride + c;
  const unsigned lo = codes4(y[0], y[1], y[2], y[3], inverse);
  if constexpr (!WIDE) {
    const int n = (int)p.cols - (int)c;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (32 * i < n) out[32 * i] = (uint8_t)(lo >> 8 * i);
  } else if constexpr (V == 8) {
    *reinterpret_cast<uint2*>(out) = make_uint2(lo, codes4(y[V - 4], y[V - 3], y[V - 2], y[V - 1], inverse));
  } else {
    *reinterpret_cast<unsigned*>(out) = lo;
  }
}

// NU units of a row per thread at once; LONG: rows of more, read twice.  The sum
// with the residual is rounded to the type it is stored in before its norm is
// taken: the backward pass, which reads what was stored, is then that of the
// very values the norm saw.
template <typename T, bool WIDE, int NU, bool LONG>
__global__ void __launch_bounds__(LONG ? 1024 : 512) forward_kernel(const RmsForwardParams p) {
  constexpr int V = kUnit<T, WIDE>;
  __shared__ float words[32];
  wait_for_predecessors();
  let_successor_start();
  const unsigned threads = p.threads, group = threadIdx.x / threads, tid = threadIdx.x - group * threads;
  const u64 row = (u64)blockIdx.x * (blockDim.x / threads) + group;
  const bool there = row < p.rows;
  const unsigned cols = there ? p.cols : 0, turn = threads * NU * V;
  const T* x = static_cast<const T*>(p.x) + row * p.x_stride;
  const T* r = static_cast<const T*>(p.residual) + row * p.residual_stride;
  T* added = static_cast<T*>(p.added) + row * p.added_stride;
  T* y = static_cast<T*>(p.y) + row * p.y_stride;

  float h[NU][V], sum = 0.f;
  for (unsigned from = 0; from < (LONG ? p.cols : 1); from += turn) {
#pragma unroll
    for (int k = 0; k < NU; ++k) load<T, WIDE>(x, from + column<T, WIDE>(tid, threads, k), cols, h[k]);
    if (p.residual) {
      float b[NU][V];
#pragma unroll
      for (int k = 0; k < NU; ++k) load<T, WIDE>(r, from + column<T, WIDE>(tid, threads, k), cols, b[k]);
#pragma unroll
      for (int k = 0; k < NU; ++k) {
#pragma unroll
        for (int i = 0; i < V; ++i) h[k][i] = rounded<T>(h[k][i] + b[k][i]);
        if (LONG) store<T, WIDE>(added, from + column<T, WIDE>(tid, threads, k), cols, h[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < NU; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) sum = fmaf(h[k][i], h[k][i], sum);
  }
  sum = row_sum(sum, words, threads);
  const float rstd = 1.f / sqrtf(sum / (float)p.cols + p.eps);
  if (p.rstd && tid == 0 && there) p.rstd[row] = rstd;
  for (unsigned from = 0; from < (LONG ? p.cols : 1); from += turn) {
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const unsigned c = from + column<T, WIDE>(tid, threads, k);
      if (LONG)
        load<T, WIDE>(p.residual ? added : x, c, cols, h[k]);
      else if (p.residual)
        store<T, WIDE>(added, c, cols, h[k]);
      float g[V];
      load_gamma<WIDE>(p.gamma, p.gamma_bf16, c, cols, g);
#pragma unroll
      for (int i = 0; i < V; ++i) h[k][i] = h[k][i] * rstd * g[i];
      if (p.y) store<T, WIDE>(y, c, cols, h[k]);
      if (p.y8) store8<T, WIDE>(p, row, there, c, h[k]);
    }
  }
}

// ---- backward: 16 bytes on their way into shared memory, the first n of them (zeros after)
__device__ __forceinline__ void copy_async16(unsigned smem, const void* gmem, int n) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(n) : "memory");
}
__device__ __forceinline__ void copies_made() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the newest n groups of this thread's copies have landed, for n up to 2
__device__ __forceinline__ void wait_copies(int n) {
  if (n == 0)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  else if (n == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 2;" ::: "memory");
}
template <typename T, int V>
__device__ __forceinline__ void load_landed(unsigned smem, float (&f)[V]) {
  unsigned w[4];
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(smem) : "memory");
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (sizeof(T) == 4) {
      f[i] = __uint_as_float(w[i]);
    } else {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// A narrow row's room in shared memory: as it lies in memory, from the 16-byte
// piece in which it begins.
template <typename T>
__host__ __device__ constexpr unsigned room_of(unsigned cols) {
  return (cols * (unsigned)sizeof(T) + 15u + 15u) / 16u * 16u;
}
// Its pieces on their way there, by the row's threads.  (A first piece that
// begins before the matrix: its elements go one by one.)
template <typename T>
__device__ __forceinline__ void bring_row(unsigned smem, const void* matrix, u64 row, u64 stride, unsigned cols, unsigned tid, unsigned threads) {
  const T* p = static_cast<const T*>(matrix) + row * stride;
  const unsigned shift = (unsigned)(reinterpret_cast<uintptr_t>(p) & 15u), bytes = shift + cols * (unsigned)sizeof(T);
  const char* from = reinterpret_cast<const char*>(p) - shift;
  for (unsigned at = 16 * tid; at < bytes; at += 16 * threads) {
    if (at == 0 && row * stride * sizeof(T) < shift) {
      for (unsigned j = 0; j < cols && shift + j * sizeof(T) < 16; ++j) {
        if constexpr (sizeof(T) == 4)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(smem + shift + 4 * j), "f"(p[j]) : "memory");
        else
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(smem + shift + 2 * j), "h"(reinterpret_cast<const unsigned short*>(p)[j]) : "memory");
      }
    } else {
      copy_async16(smem + at, from + at, (int)min(16u, bytes - at));
    }
  }
}
// A unit of it: four elements 32 columns apart, zeros past the row's end (where
// nothing is read: a row's threads may have units behind its room).  at: its
// first in shared memory; n columns are left from there.
template <typename T>
__device__ __forceinline__ void load_landed_narrow(unsigned at, int n, float (&f)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = 0.f;
    if (32 * i >= n) continue;
    if constexpr (sizeof(T) == 4) {
      asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f[i]) : "r"(at + 128 * i) : "memory");
    } else {
      unsigned short v;
      asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at + 64 * i) : "memory");
      f[i] = __uint_as_float((unsigned)v << 16);
    }
  }
}

// A group of threads keeps its columns through all its rows and adds their part
// of dgamma up in registers; the CTA's groups leave one row of partial sums.
// The rows of the next turns are on their way into shared memory while this
// turn's are in work (16384 x 5120 bf16 with dadded: 240 us without, 107 with it,
// 0.93 of the copy rate).  WIDE: each thread's units into places of its own.
// Narrow rows lie there as in memory, copied by other threads than read them (by
// plain loads 12000 x 4097 bf16 took 543 us).  Registers are bounded so that two
// CTAs or more are there to fill each other's waits for their rows' sums (one of
// 121 registers: 133 us).
template <typename T, bool WIDE, int NU, bool LARGE>
__global__ void __launch_bounds__(LARGE ? 512 : 384, LARGE && NU * kUnit<T, WIDE> >= 16 ? 1 : 2) backward_kernel(const RmsBackwardParams p) {
  constexpr int V = kUnit<T, WIDE>;
  __shared__ float words[2][16];
  extern __shared__ __align__(16) uint8_t raw[];
  wait_for_predecessors();
  let_successor_start();
  const unsigned threads = p.threads, groups = blockDim.x / threads, group = threadIdx.x / threads, tid = threadIdx.x - group * threads;
  const unsigned room = room_of<T>(p.cols);                                 // narrow: of a row
  const unsigned unit_bytes = blockDim.x * 16, stage_bytes = WIDE ? 3 * NU * unit_bytes : 3 * groups * room;
  const unsigned ring = (unsigned)__cvta_generic_to_shared(raw) + (WIDE ? threadIdx.x * 16 : 3 * group * room);
  const u64 step = (u64)gridDim.x * groups;
  u64 row = (u64)blockIdx.x * groups + group;
  auto bring = [&](u64 r, unsigned at) {   // row r into the stage at `at`
    const bool there = r < p.rows;
    if constexpr (WIDE) {
#pragma unroll
      for (int k = 0; k < NU; ++k) {
        const unsigned c = column<T, WIDE>(tid, threads, k);
        const bool mine = there && c < p.cols;
        copy_async16(at + k * unit_bytes, static_cast<const T*>(p.dy) + (mine ? r * p.dy_stride + c : 0), mine ? 16 : 0);
        copy_async16(at + (NU + k) * unit_bytes, static_cast<const T*>(p.h) + (mine ? r * p.h_stride + c : 0), mine ? 16 : 0);
        if (p.dadded) copy_async16(at + (2 * NU + k) * unit_bytes, static_cast<const T*>(p.dadded) + (mine ? r * p.dadded_stride + c : 0), mine ? 16 : 0);
      }
    } else if (there) {
      bring_row<T>(at, p.dy, r, p.dy_stride, p.cols, tid, threads);
      bring_row<T>(at + room, p.h, r, p.h_stride, p.cols, tid, threads);
      if (p.dadded) bring_row<T>(at + 2 * room, p.dadded, r, p.dadded_stride, p.cols, tid, threads);
    }
    copies_made();
  };
  // unit k of the row's dy (which 0), h (1) or dadded (2), in the stage at `at`
  auto landed = [&](unsigned at, int which, int k, const void* matrix, u64 stride, unsigned cols, float (&f)[V]) {
    if constexpr (WIDE) {
      load_landed<T>(at + (which * NU + k) * unit_bytes, f);
    } else {
      const unsigned c = column<T, WIDE>(tid, threads, k);
      const unsigned shift = (unsigned)(reinterpret_cast<uintptr_t>(static_cast<const T*>(matrix) + row * stride) & 15u);
      load_landed_narrow<T>(at + which * room + shift + c * (unsigned)sizeof(T), (int)cols - (int)c, f);
    }
  };
  constexpr bool kKeep = NU * V <= 16;   // gamma in registers; else it is read for each row
  float acc[NU][V], gamma[kKeep ? NU : 1][V];
#pragma unroll
  for (int k = 0; k < NU; ++k) {
    if constexpr (kKeep) load_gamma<WIDE>(p.gamma, p.gamma_bf16, column<T, WIDE>(tid, threads, k), p.cols, gamma[k]);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[k][i] = 0.f;
  }
  for (int s = 0; s + 1 < p.stages; ++s) bring(row + s * step, ring + s * stage_bytes);
  const float inv_cols = 1.f / (float)p.cols;
  float rstd = row < p.rows ? p.rstd[row] : 0.f;
  int buf = 0, stage = 0;
  const int ahead = p.stages - 1;
  for (u64 first = (u64)blockIdx.x * groups; first < p.rows; first += step, row += step, buf ^= 1) {
    const unsigned cols = row < p.rows ? p.cols : 0;
    const float next_rstd = row + step < p.rows ? p.rstd[row + step] : 0.f;
    const unsigned at = ring + stage * stage_bytes, into = ring + (stage == 0 ? ahead : stage - 1) * stage_bytes;
    if constexpr (WIDE) {
      bring(row + ahead * step, into);
      wait_copies(ahead);
    } else {   // what all threads copied is there, and nobody reads the stage that is filled next
      wait_copies(ahead - 1);
      __syncthreads();
      bring(row + ahead * step, into);
    }
    stage = stage == ahead ? 0 : stage + 1;
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      float x[V], y[V], (&g)[V] = gamma[kKeep ? k : 0];
      if constexpr (!kKeep) load_gamma<WIDE>(p.gamma, p.gamma_bf16, column<T, WIDE>(tid, threads, k), p.cols, g);
      landed(at, 0, k, p.dy, p.dy_stride, cols, y);
      landed(at, 1, k, p.h, p.h_stride, cols, x);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[i] *= rstd;
        acc[k][i] = fmaf(y[i], x[i], acc[k][i]);
        sum = fmaf(y[i] * g[i], x[i], sum);
      }
    }
    sum = row_sum(sum, words[buf], threads) * inv_cols;
    T* dx = static_cast<T*>(p.dx) + row * p.dx_stride;
#pragma unroll
    for (int k = 0; k < NU; ++k) {   // (read once more: registers for them would cost a CTA)
      float x[V], y[V], e[V], (&g)[V] = gamma[kKeep ? k : 0];
      if constexpr (!kKeep) load_gamma<WIDE>(p.gamma, p.gamma_bf16, column<T, WIDE>(tid, threads, k), p.cols, g);
      landed(at, 0, k, p.dy, p.dy_stride, cols, y);
      landed(at, 1, k, p.h, p.h_stride, cols, x);
      if (p.dadded) landed(at, 2, k, p.dadded, p.dadded_stride, cols, e);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        y[i] = fmaf(-(x[i] * rstd), sum, y[i] * g[i]) * rstd;
        if (p.dadded) y[i] += e[i];
      }
      store<T, WIDE>(dx, column<T, WIDE>(tid, threads, k), cols, y);
    }
    rstd = next_rstd;
  }
  wait_copies(0);
  if (!p.partial) return;
  float* mine = p.partial + (u64)blockIdx.x * p.cols;
  if (groups > 1) {
    float* parts = reinterpret_cast<float*>(raw);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < NU; ++k)
#pragma unroll
      for (int i = 0; i < V; ++i) parts[(group * NU * V + k * V + i) * threads + tid] = acc[k][i];
    __syncthreads();
    if (group) return;
    for (unsigned j = 1; j < groups; ++j)
#pragma unroll
      for (int k = 0; k < NU; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[k][i] += parts[(j * NU * V + k * V + i) * threads + tid];
  }
#pragma unroll
  for (int k = 0; k < NU; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const unsigned c = column<T, WIDE>(tid, threads, k) + kApart<WIDE> * i;
      if (c < p.cols) mine[c] = acc[k][i];
    }
}

// Long rows, first launch: sum(a * xhat) / cols of each row.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(1024) long_sums_kernel(const RmsBackwardParams p) {
  constexpr int V = kUnit<T, WIDE>;
  __shared__ float words[32];
  wait_for_predecessors();
  let_successor_start();
  const u64 row = blockIdx.x;
  const T* dy = static_cast<const T*>(p.dy) + row * p.dy_stride;
  const T* x = static_cast<const T*>(p.h) + row * p.h_stride;
  const float rstd = p.rstd[row];
  float sum = 0.f;
  for (unsigned from = 0; from < p.cols; from += blockDim.x * V) {
    const unsigned c = from + column<T, WIDE>(threadIdx.x, blockDim.x, 0);
    float d[V], h[V], g[V];
    load<T, WIDE>(dy, c, p.cols, d);
    load<T, WIDE>(x, c, p.cols, h);
    load_gamma<WIDE>(p.gamma, p.gamma_bf16, c, p.cols, g);
#pragma unroll
    for (int i = 0; i < V; ++i) sum = fmaf(d[i] * g[i], h[i] * rstd, sum);
  }
  sum = row_sum(sum, words, blockDim.x);
  if (threadIdx.x == 0) p.row_sums[row] = sum / (float)p.cols;
}
// Second launch: a CTA takes a slice of the columns through every gridDim.y-th row.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(256) long_rows_kernel(const RmsBackwardParams p) {
  constexpr int V = kUnit<T, WIDE>;
  wait_for_predecessors();
  let_successor_start();
  const unsigned c = blockIdx.x * blockDim.x * V + column<T, WIDE>(threadIdx.x, blockDim.x, 0);
  float acc[V], g[V];
  load_gamma<WIDE>(p.gamma, p.gamma_bf16, c, p.cols, g);
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll 2
  for (u64 row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const float rstd = p.rstd[row], sum = p.row_sums[row];
    float d[V], h[V], e[V];
    load<T, WIDE>(static_cast<const T*>(p.dy) + row * p.dy_stride, c, p.cols, d);
    load<T, WIDE>(static_cast<const T*>(p.h) + row * p.h_stride, c, p.cols, h);
    if (p.dadded) load<T, WIDE>(static_cast<const T*>(p.dadded) + row * p.dadded_stride, c, p.cols, e);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      h[i] *= rstd;
      acc[i] = fmaf(d[i], h[i], acc[i]);
      d[i] = fmaf(-h[i], sum, d[i] * g[i]) * rstd;
      if (p.dadded) d[i] += e[i];
    }
    store<T, WIDE>(static_cast<T*>(p.dx) + row * p.dx_stride, c, p.cols, d);
  }
  if (!p.partial) return;
  float* mine = p.partial + (u64)blockIdx.y * p.cols;
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (c + kApart<WIDE> * i < p.cols) mine[c + kApart<WIDE> * i] = acc[i];
}

// dgamma from the partial sums: 16 columns (two sectors of a row of them) per
// CTA, every 32nd row by the same 16 threads.
constexpr int kSumCols = 16, kSumRows = 32;
__global__ void __launch_bounds__(kSumCols * kSumRows) sum_parts_kernel(const RmsBackwardParams p) {
  __shared__ float words[kSumRows][kSumCols + 1];
  wait_for_predecessors();
  let_successor_start();
  const unsigned at = threadIdx.x / kSumCols, i = threadIdx.x % kSumCols, c = blockIdx.x * kSumCols + i;
  float v = 0.f;
  if (c < p.cols) {
#pragma unroll 8
    for (unsigned j = at; j < p.nparts; j += kSumRows) v += p.partial[(u64)j * p.cols + c];
  }
  words[at][i] = v;
  __syncthreads();
  const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = warp_sum(words[lane][warp]);   // 16 warps, 32 rows
  const unsigned out = blockIdx.x * kSumCols + warp;
  if (lane == 0 && out < p.cols) p.dgamma[out] = p.accumulate ? p.dgamma[out] + v : v;
}

unsigned round32(u64 n) { return (unsigned)((n + 31) / 32 * 32); }

template <typename T, bool WIDE>
cudaError_t forward(RmsForwardParams& p, cudaStream_t st) {
  constexpr int V = kUnit<T, WIDE>;
  const unsigned units = WIDE ? (p.cols + V - 1) / V : (p.cols + 127) / 128 * 32;
  if (units > 4 * 512) {
    p.threads = 1024;
    return launch_dependent(forward_kernel<T, WIDE, 2, true>, dim3((unsigned)p.rows), 1024, 0, 1, st, p);
  }
  // Two units a thread where a row has more than a warp's, so that a row's own steps are shared by more elements, and four
  // in long rows (bf16, with the residual: 16384 x 2048 47 us by two and 63 by one, 6000 x 8192 69 by four and 73 by two;
  // unaligned rows 98 by two and 116 by four at 16384 x 2049).
  const unsigned nu = units <= 32 ? 1 : units <= (WIDE ? 512 : 1024) ? 2 : 4;
  p.threads = round32((units + nu - 1) / nu);
  const unsigned groups = p.threads >= 128 ? 1 : 128 / p.threads;
  const dim3 grid((unsigned)((p.rows + groups - 1) / groups));
  const int block = (int)(groups * p.threads);
  switch (nu) {
    case 1: return launch_dependent(forward_kernel<T, WIDE, 1, false>, grid, block, 0, 1, st, p);
    case 2: return launch_dependent(forward_kernel<T, WIDE, 2, false>, grid, block, 0, 1, st, p);
    default: return launch_dependent(forward_kernel<T, WIDE, 4, false>, grid, block, 0, 1, st, p);
  }
}

template <typename T, bool WIDE, int NU>
cudaError_t backward_rows(RmsBackwardParams& p, const RmsBackwardShape& s, cudaStream_t st) {
  const unsigned block = s.groups * s.threads, stage = WIDE ? 3 * NU * 16 * block : 3 * s.groups * room_of<T>(p.cols);
  // As many rows ahead as the SM's CTAs have room for: two at most where units are wide (16384 x 8192 bf16 with dadded 176 us,
  // 180 by three; 60000 x 256 24.3 and 25.8), else three, the first of which has to be there a turn early.
  p.stages = std::min(WIDE ? 3 : 4, std::max(2, (int)(200 * 1024 / (s.per_sm * stage))));
  size_t smem = (size_t)p.stages * stage;
  if (s.groups > 1) smem = std::max<size_t>(smem, (size_t)block * NU * kUnit<T, WIDE> * sizeof(float));
  constexpr bool kSmall = (!WIDE && NU <= 2) || NU * kUnit<T, WIDE> > 16;   // 64 registers do, or 128 are needed, in CTAs of any size
  const auto kernel = block > 384 ? backward_kernel<T, WIDE, NU, true> : backward_kernel<T, WIDE, NU, kSmall>;
  return launch_dependent(kernel, dim3(s.nparts), (int)block, smem, 1, st, p);
}

template <typename T, bool WIDE>
cudaError_t backward(RmsBackwardParams& p, const RmsBackwardShape& s, cudaStream_t st) {
  constexpr int V = kUnit<T, WIDE>;
  p.threads = s.threads;
  p.nparts = s.nparts;
  cudaError_t e;
  if (s.is_long) {
    e = launch_dependent(long_sums_kernel<T, WIDE>, dim3((unsigned)p.rows), 1024, 0, 1, st, p);
    if (e != cudaSuccess) return e;
    e = launch_dependent(long_rows_kernel<T, WIDE>, dim3((p.cols + 256 * V - 1) / (256 * V), s.nparts), 256, 0, 1, st, p);
  } else {
    e = s.nu == 1 ? backward_rows<T, WIDE, 1>(p, s, st) : s.nu == 2 ? backward_rows<T, WIDE, 2>(p, s, st) : backward_rows<T, WIDE, 4>(p, s, st);
  }
  if (e != cudaSuccess || !p.dgamma) return e;
  return launch_dependent(sum_parts_kernel, dim3((p.cols + kSumCols - 1) / kSumCols), kSumCols * kSumRows, 0, 1, st, p);
}

}  // namespace

RmsBackwardShape rms_backward_shape(size_t rows, size_t cols, int dtype, bool wide, int sms) {
  const unsigned v = wide && dtype == XP_BF16 ? 8 : 4;
  const unsigned units = wide ? (unsigned)((cols + v - 1) / v) : (unsigned)((cols + 127) / 128 * 32);
  RmsBackwardShape s = {};
  // More than one unit a thread where a row has more than a warp's: 16384 x 2048 bf16 47 us by two and 54 by one, 60000 x 512
  // 41, 48 and by four 74; unaligned rows 60000 x 257 bf16 67 by four, 79 by two and 98 by one, 16384 x 2049 101 by four and
  // 108 by two, but 4099 x 1031 fp32 18 by two and 20 by four.
  s.nu = units <= 32 ? 1 : !wide && (units <= 128 || dtype == XP_BF16) ? 4 : units <= 1024 ? 2 : 4;
  s.threads = round32((units + s.nu - 1) / s.nu);
  s.is_long = s.threads > 512;
  if (s.is_long) {
    const size_t slices = (cols + 256 * v - 1) / (256 * v), most = (8 * (size_t)sms + slices - 1) / slices;
    s.nparts = (unsigned)std::min<size_t>(rows, std::max<size_t>(1, most));
    return s;
  }
  s.groups = s.threads >= 256 ? 1 : 256 / s.threads;
  const unsigned block = s.groups * s.threads;
  // by their registers, of which a quarter of the SM gives each of its warps a whole number: 128 a thread where it keeps
  // 32 columns' sums, or 16 in CTAs of more than 384 threads, 80 in smaller ones, else 64
  const unsigned regs = s.nu * v == 32 ? 128 : !wide && s.nu <= 2 ? 64 : block <= 384 ? 80 : s.nu * v == 16 ? 128 : 64;
  const unsigned es = dtype == XP_F32 ? 4 : 2, stage = wide ? 3 * s.nu * 16 * block : 3 * s.groups * (es == 4 ? room_of<float>((unsigned)cols) : room_of<bf16>((unsigned)cols));
  s.per_sm = std::min(4 * (512 / regs) / (block / 32), 216 * 1024 / (2 * stage));   // two rows each in shared memory
  s.per_sm = std::max(1u, s.per_sm);
  s.nparts = (unsigned)std::min<size_t>((rows + s.groups - 1) / s.groups, (size_t)sms * s.per_sm);
  return s;
}

cudaError_t launch_rms_forward(RmsForwardParams& p, int dtype, bool wide, cudaStream_t st) {
  if (dtype == XP_F32) return wide ? forward<float, true>(p, st) : forward<float, false>(p, st);
  return wide ? forward<bf16, true>(p, st) : forward<bf16, false>(p, st);
}

cudaError_t launch_rms_backward(RmsBackwardParams& p, const RmsBackwardShape& s, int dtype, bool wide, cudaStream_t st) {
  if (dtype == XP_F32) return wide ? backward<float, true>(p, s, st) : backward<float, false>(p, s, st);
  return wide ? backward<bf16, true>(p, s, st) : backward<bf16, false>(p, s, st);
}

}  // namespace xp
