// Matrices to and from 8 bits by blocks of 128 (include/xp_model.h).
//
// HBM bounds both directions: an element is read once and each of its codes
// written once.  An encoding CTA takes 128 x 128 elements into registers, so
// that a block's scale is known before its codes, along rows and along columns
// alike; the transposed codes go through shared memory.
#include "xp_code8.cuh"
#include "xp_model_internal.h"
#include "xp_train_device.cuh"

namespace xp {
namespace {

typedef __nv_bfloat16 bf16;
typedef unsigned long long u64;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTurns = 128 / (4 * kWarps);   // a warp takes 4 rows at a time

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }

// n of 4 neighbouring elements; zeros behind them
template <typename T>
__device__ __forceinline__ void load4(const T* p, int n, bool aligned, float (&f)[4]) {
  if (n >= 4 && aligned) {
    if constexpr (sizeof(T) == 4) {
      const float4 q = *reinterpret_cast<const float4*>(p);
      f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
    } else {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      f[0] = __uint_as_float(q.x << 16), f[1] = __uint_as_float(q.x & 0xffff0000u);
      f[2] = __uint_as_float(q.y << 16), f[3] = __uint_as_float(q.y & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < n ? to_f(p[i]) : 0.f;
  }
}
__device__ __forceinline__ void store4(uint8_t* p, unsigned codes, int n, bool aligned) {
  if (n >= 4 && aligned) {
    *reinterpret_cast<unsigned*>(p) = codes;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = (uint8_t)(codes >> 8 * i);
  }
}

// Rows of the tile: warp w has 4 w .. 4 w + 3 of each 32 (turn), lane l the
// columns 4 l .. 4 l + 3.  So four rows' codes of a column are one word of the
// transposed tile, whose word (column, rows / 4) is kept at the place that
// column / 4 turns: a warp's words lie in 32 banks when it writes those of a
// row and when it reads those of a column.
template <typename T, bool TILE>
__global__ void __launch_bounds__(kThreads) encode_kernel(const Encode8Params p) {
  __shared__ unsigned words[128 * 32];
  __shared__ unsigned tops[kWarps][128];
  wait_for_predecessors();
  let_successor_start();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned tile_r = blockIdx.x / p.tiles_c, tile_c = blockIdx.x - tile_r * p.tiles_c;
  const unsigned r0 = tile_r * 128, c0 = tile_c * 128 + 4 * lane;
  const int n = (int)min(4u, p.cols > c0 ? p.cols - c0 : 0u);
  const T* x = static_cast<const T*>(p.x) + (u64)r0 * p.x_stride + c0;
  float f[kTurns][4][4];
#pragma unroll
  for (int t = 0; t < kTurns; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const unsigned r = 32 * t + 4 * warp + i;
      load4(x + r * p.x_stride, r0 + r < p.rows ? n : 0, p.x_aligned, f[t][i]);
    }

  unsigned tile_e = 0;
  if (TILE || p.codes_t) {
    unsigned top[4] = {0, 0, 0, 0};
#pragma unroll
    for (int t = 0; t < kTurns; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) top[c] = max(top[c], abs_bits(f[t][i][c]));
    if constexpr (TILE) {
      const unsigned all = __reduce_max_sync(0xffffffffu, max(max(top[0], top[1]), max(top[2], top[3])));
      if (lane == 0) tops[warp][0] = all;
      __syncthreads();
      unsigned most = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) most = max(most, tops[w][0]);
      tile_e = scale_of(most);
      if (threadIdx.x == 0) {
        if (p.codes) p.scales[tile_r * p.scales_stride + tile_c] = (uint8_t)tile_e;
        if (p.codes_t) p.scales_t[tile_c * p.scales_t_stride + tile_r] = (uint8_t)tile_e;
      }
    } else {
      *reinterpret_cast<uint4*>(&tops[warp][4 * lane]) = make_uint4(top[0], top[1], top[2], top[3]);
      __syncthreads();
    }
  }

  if (p.codes) {
    uint8_t* codes = p.codes + (u64)r0 * p.codes_stride + c0;
#pragma unroll
    for (int t = 0; t < kTurns; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const unsigned r = 32 * t + 4 * warp + i;
        const float(&v)[4] = f[t][i];
        unsigned e = tile_e;
        if constexpr (!TILE) {
          e = scale_of(__reduce_max_sync(0xffffffffu, max(max(abs_bits(v[0]), abs_bits(v[1])), max(abs_bits(v[2]), abs_bits(v[3])))));
          if (lane == 0 && r0 + r < p.rows) p.scales[(u64)(r0 + r) * p.scales_stride + tile_c] = (uint8_t)e;
        }
        store4(codes + r * p.codes_stride, codes4(v[0], v[1], v[2], v[3], inverse_of(e), e), r0 + r < p.rows ? n : 0, p.codes_aligned);
      }
  }
  if (!p.codes_t) return;

#pragma unroll
  for (int c = 0; c < 4; ++c) {
    unsigned e = tile_e;
    if constexpr (!TILE) {
      unsigned most = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) most = max(most, tops[w][4 * lane + c]);
      e = scale_of(most);
      if (warp == 0 && c < n) p.scales_t[(u64)(c0 + c) * p.scales_t_stride + tile_r] = (uint8_t)e;
    }
    const float inverse = inverse_of(e);
#pragma unroll
    for (int t = 0; t < kTurns; ++t)
      words[(4 * lane + c) * 32 + ((kWarps * t + warp) ^ lane)] = codes4(f[t][0][c], f[t][1][c], f[t][2][c], f[t][3][c], inverse, e);
  }
  __syncthreads();
  const unsigned row = r0 + 4 * lane;
  const int nr = (int)min(4u, p.rows > row ? p.rows - row : 0u);
#pragma unroll
  for (int j = 0; j < 128 / kWarps; ++j) {
    const unsigned c = warp * (128 / kWarps) + j, col = tile_c * 128 + c;
    if (col < p.cols) store4(p.codes_t + (u64)col * p.codes_t_stride + row, words[c * 32 + (lane ^ (c >> 2))], nr, p.codes_t_aligned);
  }
}

// 16 codes per thread; a row's threads side by side.
template <typename T>
__global__ void __launch_bounds__(kThreads) decode_kernel(const Decode8Params p) {
  wait_for_predecessors();
  let_successor_start();
  const unsigned per_row = (p.cols + 15) / 16;
  const u64 at = (u64)blockIdx.x * kThreads + threadIdx.x;
  if (at >= (u64)per_row * p.rows) return;
  const unsigned row = (unsigned)(at / per_row), c = ((unsigned)(at - (u64)row * per_row)) * 16;
  const int n = (int)min(16u, p.cols - c);
  const uint8_t* from = p.codes + (u64)row * p.codes_stride + c;
  T* out = static_cast<T*>(p.out) + (u64)row * p.out_stride + c;
  const float scale = power_of(p.scales[(u64)(row >> p.shift) * p.scales_stride + c / 128]);
  if (n == 16 && p.aligned) {
    const uint4 q = *reinterpret_cast<const uint4*>(from);
    const unsigned w[4] = {q.x, q.y, q.z, q.w};
    float v[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 f = values2((unsigned short)(w[i / 2] >> 16 * (i & 1)));
      v[2 * i] = f.x * scale;
      v[2 * i + 1] = f.y * scale;
    }
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) reinterpret_cast<float4*>(out)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        unsigned u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]);
          u[j] = *reinterpret_cast<const unsigned*>(&h);
        }
        reinterpret_cast<uint4*>(out)[i] = make_uint4(u[0], u[1], u[2], u[3]);
      }
    }
    return;
  }
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float v = values2(from[i]).x * scale;
    if constexpr (sizeof(T) == 4)
      out[i] = v;
    else
      out[i] = __float2bfloat16_rn(v);
  }
}

}  // namespace

cudaError_t launch_encode8(const Encode8Params& p, int dtype, int block_rows, cudaStream_t st) {
  const u64 tiles = (u64)p.tiles_c * ((p.rows + 127) / 128);
  const auto kernel = dtype == XP_F32 ? (block_rows == 1 ? encode_kernel<float, false> : encode_kernel<float, true>)
                                      : (block_rows == 1 ? encode_kernel<bf16, false> : encode_kernel<bf16, true>);
  return launch_dependent(kernel, dim3((unsigned)tiles), kThreads, 0, 1, st, p);
}

cudaError_t launch_decode8(const Decode8Params& p, int dtype, cudaStream_t st) {
  const u64 n = (u64)((p.cols + 15) / 16) * p.rows;
  return launch_dependent(dtype == XP_F32 ? decode_kernel<float> : decode_kernel<bf16>, dim3((unsigned)((n + kThreads - 1) / kThreads)), kThreads, 0, 1, st, p);
}

}  // namespace xp
