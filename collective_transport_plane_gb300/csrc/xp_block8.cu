// Matrices to and from 8 bits by blocks of 128 (include/xp_model.h).
//
// HBM bounds both directions: an element is read once and each of its codes
// written once.  An encoding CTA takes 128 x 128 elements into registers, so
// that a block's scale is known before its codes, along rows and along columns
// alike; the transposed codes go through shared memory.
#include "xp_code8.cuh"
#include "xp_fours.cuh"
#include "xp_model_internal.h"
#include "xp_train_device.cuh"

namespace xp {
namespace {

typedef __nv_bfloat16 bf16;
typedef unsigned long long u64;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kTurns = 128 / (4 * kWarps);   // a warp takes 4 rows at a time

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }

// Four neighbouring elements as they are stored: registers decide how many CTAs an SM has.
template <typename T>
struct Four;
template <>
struct Four<float> {
  float4 q;
  __device__ __forceinline__ void load(const float* p) { q = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void set(const float (&f)[4]) { q = make_float4(f[0], f[1], f[2], f[3]); }
  __device__ __forceinline__ void get(float (&f)[4]) const { f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w; }
  // Largest magnitudes, of each of the four columns or of all: as bits, NaN above all.
  struct Tops {
    unsigned t[4] = {0, 0, 0, 0};
  };
  __device__ __forceinline__ void raise(Tops& m) const {
    m.t[0] = max(m.t[0], abs_bits(q.x)), m.t[1] = max(m.t[1], abs_bits(q.y));
    m.t[2] = max(m.t[2], abs_bits(q.z)), m.t[3] = max(m.t[3], abs_bits(q.w));
  }
  static __device__ __forceinline__ uint4 tops(const Tops& m) { return make_uint4(m.t[0], m.t[1], m.t[2], m.t[3]); }
  __device__ __forceinline__ unsigned top() const { return max(max(abs_bits(q.x), abs_bits(q.y)), max(abs_bits(q.z), abs_bits(q.w))); }
};
template <>
struct Four<bf16> {
  uint2 q;
  __device__ __forceinline__ void load(const bf16* p) { q = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void set(const float (&f)[4]) {   // exact: these were bf16
    q.x = __float_as_uint(f[0]) >> 16 | (__float_as_uint(f[1]) & 0xffff0000u);
    q.y = __float_as_uint(f[2]) >> 16 | (__float_as_uint(f[3]) & 0xffff0000u);
  }
  __device__ __forceinline__ void get(float (&f)[4]) const {
    f[0] = __uint_as_float(q.x << 16), f[1] = __uint_as_float(q.x & 0xffff0000u);
    f[2] = __uint_as_float(q.y << 16), f[3] = __uint_as_float(q.y & 0xffff0000u);
  }
  struct Tops {   // two columns' in a word; NaN above all
    unsigned t[2] = {0, 0};
  };
  static __device__ __forceinline__ unsigned larger(unsigned m, unsigned w) {
    const __nv_bfloat162 a = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&m), __habs2(*reinterpret_cast<const __nv_bfloat162*>(&w)));
    return *reinterpret_cast<const unsigned*>(&a);
  }
  __device__ __forceinline__ void raise(Tops& m) const { m.t[0] = larger(m.t[0], q.x), m.t[1] = larger(m.t[1], q.y); }
  static __device__ __forceinline__ uint4 tops(const Tops& m) { return make_uint4(m.t[0] << 16, m.t[0] & 0xffff0000u, m.t[1] << 16, m.t[1] & 0xffff0000u); }
  __device__ __forceinline__ unsigned top() const {
    const unsigned m = larger(q.x & 0x7fff7fffu, q.y);
    return max(m << 16, m & 0xffff0000u);
  }
};
// n of them; zeros behind
template <typename T>
__device__ __forceinline__ Four<T> load4(const T* p, int n, bool aligned) {
  Four<T> four;
  if (n >= 4 && aligned) {
    four.load(p);
  } else {
    float f[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < n ? to_f(p[i]) : 0.f;
    four.set(f);
  }
  return four;
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

// Rows of the tile: warp w has 4 w .. 4 w + 3 of each 64 (turn), lane l the
// columns 4 l .. 4 l + 3.  So four rows' codes of a column are one word of the
// transposed tile, whose word (column, rows / 4) is kept at the place that
// column / 4 turns: a warp's words lie in 32 banks when it writes those of a
// row and when it reads those of a column.
// A thread's 4 elements of each of its rows on their way into shared memory, into places of its own.
template <typename T>
__device__ __forceinline__ unsigned place_of(const uint8_t* ahead, int t, int i) {
  return (unsigned)__cvta_generic_to_shared(ahead) + (unsigned)((t * 4 + i) * kThreads + threadIdx.x) * 4 * (unsigned)sizeof(T);
}
template <typename T>
__device__ __forceinline__ void bring_tile(const Encode8Params& p, const uint8_t* ahead, unsigned tile_r, unsigned tile_c) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const T* x = static_cast<const T*>(p.x) + (u64)(tile_r * 128 + 4 * warp) * p.x_stride + tile_c * 128 + 4 * lane;
#pragma unroll
  for (int t = 0; t < kTurns; ++t, x += 4 * kWarps * p.x_stride) {
    const T* at = x;
#pragma unroll
    for (int i = 0; i < 4; ++i, at += p.x_stride)
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(place_of<T>(ahead, t, i)), "l"(at), "n"(4 * (int)sizeof(T)) : "memory");
  }
}

// The piece that holds column c of a row, or none.
__device__ __forceinline__ uint2 piece_of(const Encode8Params& p, const bf16* from, unsigned row, int c) {
  if (row >= p.rows) return make_uint2(0, 0);
  return piece_at(from, c - ahead_of(from), (int)p.cols, pieces_inside(row * p.x_stride, (p.rows - 1 - row) * p.x_stride + p.cols, p.cols));
}

// WHOLE: all of the tile is there, and its rows and columns are aligned; its
// elements came ahead.  taken: called when they are in registers.
template <typename T, bool TILE, bool WHOLE, typename Taken>
__device__ __forceinline__ void encode_tile(const Encode8Params& p, unsigned (&words)[128 * 32], unsigned (&tops)[kWarps][128], const uint8_t* ahead,
                                            unsigned tile_r, unsigned tile_c, Taken taken) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned r0 = tile_r * 128, c0 = tile_c * 128 + 4 * lane;
  const int n = WHOLE ? 4 : (int)min(4u, p.cols > c0 ? p.cols - c0 : 0u);
  // this warp's rows of turn 0; a turn's are kWarps * 4 rows further
  const unsigned mine = 4 * warp, next = 4 * kWarps;
  const T* x = static_cast<const T*>(p.x) + (u64)(r0 + mine) * p.x_stride + c0;
  Four<T> four[kTurns][4];
  bool taken_by_pieces = false;
  if constexpr (sizeof(T) == 2 && !WHOLE) {
    // (element by element 12000 x 4097 took 81 us, 64 by pieces; short rows' ends cost more: 20000 x 333 10.9, 13.3 by pieces)
    taken_by_pieces = !p.x_aligned && p.cols >= 512;
    if (taken_by_pieces) {
#pragma unroll
      for (int t = 0; t < kTurns; ++t) {
        const unsigned row = r0 + mine + next * t;
        const T* from = x - c0 + next * t * p.x_stride;
        uint2 q[4], more = make_uint2(0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = piece_of(p, from + i * p.x_stride, row + i, (int)c0);
        if (lane < 4) more = piece_of(p, from + lane * p.x_stride, row + lane, (int)(tile_c * 128 + 128));   // behind the last lane's
#pragma unroll
        for (int i = 0; i < 4; ++i) four[t][i].q = join_pieces(q[i], more, i, ahead_of(from + i * p.x_stride), c0, row + i < p.rows ? p.cols : 0);
      }
    }
  }
  if (!taken_by_pieces) {
#pragma unroll
    for (int t = 0; t < kTurns; ++t, x += next * p.x_stride) {
      const T* at = x;
#pragma unroll
      for (int i = 0; i < 4; ++i, at += p.x_stride) {
        if (WHOLE)
          four[t][i].load(reinterpret_cast<const T*>(ahead) + 4 * ((t * 4 + i) * kThreads + threadIdx.x));
        else
          four[t][i] = load4(at, r0 + mine + next * t + i < p.rows ? n : 0, p.x_aligned);
      }
    }
  }

  taken();

  unsigned tile_e = 0;
  if (TILE || p.codes_t) {
    typename Four<T>::Tops most_of;
#pragma unroll
    for (int t = 0; t < kTurns; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) four[t][i].raise(most_of);
    const uint4 top = Four<T>::tops(most_of);
    if constexpr (TILE) {
      const unsigned all = __reduce_max_sync(0xffffffffu, max(max(top.x, top.y), max(top.z, top.w)));
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
      *reinterpret_cast<uint4*>(&tops[warp][4 * lane]) = top;
      __syncthreads();
      if (threadIdx.x < 128) {   // a column's scale by one thread; its inverse goes into the first warp's row
        unsigned most = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) most = max(most, tops[w][threadIdx.x]);
        const unsigned e = scale_of(most), col = tile_c * 128 + threadIdx.x;
        tops[0][threadIdx.x] = __float_as_uint(inverse_of(e));
        if (WHOLE || col < p.cols) p.scales_t[(u64)col * p.scales_t_stride + tile_r] = (uint8_t)e;
      }
      __syncthreads();
    }
  }

  const float tile_inverse = inverse_of(tile_e);
  if (p.codes) {
    uint8_t* codes = p.codes + (u64)(r0 + mine) * p.codes_stride + c0;
    uint8_t* scales = p.scales + (u64)(r0 + mine) * p.scales_stride + tile_c;
#pragma unroll
    for (int t = 0; t < kTurns; ++t, codes += next * p.codes_stride, scales += next * p.scales_stride) {
      unsigned e[4];
      if constexpr (!TILE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = scale_of(__reduce_max_sync(0xffffffffu, four[t][i].top()));
        // four rows' scales by four lanes
        const unsigned m = lane == 0 ? e[0] : lane == 1 ? e[1] : lane == 2 ? e[2] : e[3];
        if (lane < 4 && (WHOLE || r0 + mine + next * t + lane < p.rows)) scales[lane * p.scales_stride] = (uint8_t)m;
      }
      uint8_t* at = codes;
#pragma unroll
      for (int i = 0; i < 4; ++i, at += p.codes_stride) {
        float f[4];
        four[t][i].get(f);
        const unsigned c = codes4(f[0], f[1], f[2], f[3], TILE ? tile_inverse : inverse_of(e[i]));
        if (WHOLE)
          *reinterpret_cast<unsigned*>(at) = c;
        else
          store4(at, c, r0 + mine + next * t + i < p.rows ? n : 0, p.codes_aligned);
      }
    }
  }
  if (!p.codes_t) return;   // the same for the CTA

  float inverse[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) inverse[c] = TILE ? tile_inverse : __uint_as_float(tops[0][4 * lane + c]);
#pragma unroll
  for (int t = 0; t < kTurns; ++t) {
    float f[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) four[t][i].get(f[i]);
    unsigned* to = words + 128 * lane + ((kWarps * t + warp) ^ lane);
#pragma unroll
    for (int c = 0; c < 4; ++c) to[32 * c] = codes4(f[0][c], f[1][c], f[2][c], f[3][c], inverse[c]);
  }
  __syncthreads();
  const unsigned row = r0 + 4 * lane, first = warp * (128 / kWarps);
  const int nr = WHOLE ? 4 : (int)min(4u, p.rows > row ? p.rows - row : 0u);
  uint8_t* out = p.codes_t + (u64)(tile_c * 128 + first) * p.codes_t_stride + row;
#pragma unroll
  for (int j = 0; j < 128 / kWarps; ++j, out += p.codes_t_stride) {
    const unsigned c = first + j, word = words[c * 32 + (lane ^ (c >> 2))];
    if (WHOLE)
      *reinterpret_cast<unsigned*>(out) = word;
    else if (tile_c * 128 + c < p.cols)
      store4(out, word, nr, p.codes_t_aligned);
  }
}

// CTAs take tiles one after another, the next one's elements on their way
// meanwhile.  (16384 x 4096 bf16, both forms: 80 us with addresses and edges
// worked out for every row, at 30 instructions for each element; 58 without,
// a tile per CTA and nothing on its way while codes are made.)
template <typename T, bool TILE>
__global__ void __launch_bounds__(kThreads, 2) encode_kernel(const Encode8Params p) {
  extern __shared__ __align__(16) uint8_t raw[];
  auto& words = *reinterpret_cast<unsigned(*)[128 * 32]>(raw);
  auto& tops = *reinterpret_cast<unsigned(*)[kWarps][128]>(raw + sizeof words);
  const uint8_t* ahead = raw + sizeof words + sizeof tops;
  wait_for_predecessors();
  let_successor_start();
  auto whole = [&](unsigned tile, unsigned& r, unsigned& c) {
    r = tile / p.tiles_c;
    c = tile - r * p.tiles_c;
    return p.all_aligned && (r + 1) * 128 <= p.rows && (c + 1) * 128 <= p.cols;
  };
  unsigned r, c;
  if (whole(blockIdx.x, r, c)) bring_tile<T>(p, ahead, r, c);
  for (unsigned tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    const bool now = whole(tile, r, c);
    const auto next = [&] {
      unsigned nr, nc;
      if (tile + gridDim.x < p.tiles && whole(tile + gridDim.x, nr, nc)) bring_tile<T>(p, ahead, nr, nc);
    };
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (now)
      encode_tile<T, TILE, true>(p, words, tops, ahead, r, c, next);
    else
      encode_tile<T, TILE, false>(p, words, tops, ahead, r, c, next);
    __syncthreads();   // words and tops are free
  }
}

// A warp has a piece of a row.  Where rows are aligned its lanes
// take the codes of 16 bytes of output each, side by side (each lane 16 codes, in
// two stores of every other 16 bytes: 36 us for 16384 x 4096 to bf16), else every
// 32nd column.
constexpr int kDecodeThreads = 256;

template <typename T, unsigned kPiece>
__global__ void __launch_bounds__(kDecodeThreads) decode_kernel(const Decode8Params p) {
  wait_for_predecessors();
  let_successor_start();
  const int lane = threadIdx.x & 31;
  const unsigned per_row = (p.cols + kPiece - 1) / kPiece;
  const u64 piece = (u64)blockIdx.x * (kDecodeThreads / 32) + (threadIdx.x >> 5);
  if (piece >= (u64)per_row * p.rows) return;
  const u64 row = piece / per_row;
  const unsigned from = (unsigned)(piece - row * per_row) * kPiece;
  const uint8_t* codes = p.codes + row * p.codes_stride;
  const uint8_t* scales = p.scales + (row >> p.shift) * p.scales_stride;
  T* out = static_cast<T*>(p.out) + row * p.out_stride;
  constexpr int E = 16 / (int)sizeof(T), N = kPiece / 32 / E;
  if (p.aligned && p.cols % E == 0) {
    unsigned w[N][E / 4];
    float scale[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const unsigned c = from + (32 * k + lane) * E;
      if (c >= p.cols) break;
      scale[k] = power_of(scales[c / 128]);
      if constexpr (E == 8) {
        const uint2 q = *reinterpret_cast<const uint2*>(codes + c);
        w[k][0] = q.x, w[k][1] = q.y;
      } else {
        w[k][0] = *reinterpret_cast<const unsigned*>(codes + c);
      }
    }
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const unsigned c = from + (32 * k + lane) * E;
      if (c >= p.cols) break;
      float v[E];
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float2 f = values2((unsigned short)(w[k][i / 2] >> 16 * (i & 1)));
        v[2 * i] = f.x * scale[k], v[2 * i + 1] = f.y * scale[k];
      }
      if constexpr (E == 8) {
        unsigned u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
          u[j] = *reinterpret_cast<const unsigned*>(&h);
        }
        *reinterpret_cast<uint4*>(out + c) = make_uint4(u[0], u[1], u[2], u[3]);
      } else {
        *reinterpret_cast<float4*>(out + c) = make_float4(v[0], v[1], v[2], v[3]);
      }
    }
    return;
  }
  constexpr int M = kPiece >= 512 ? 16 : kPiece / 32;   // elements at a time
#pragma unroll
  for (int part = 0; part < (int)kPiece / 32 / M; ++part) {
    const unsigned c0 = from + 32 * M * part + lane;
    const int n = (int)p.cols - (int)c0;
    const uint8_t* in = codes + c0;
    T* to = out + c0;
    uint8_t code[M];
    float e[M / 4];
#pragma unroll
    for (int i = 0; i < M; ++i) {
      code[i] = 32 * i < n ? in[32 * i] : 0;
      if (i % 4 == 0) e[i / 4] = 32 * i < n ? power_of(scales[c0 / 128 + i / 4]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const float v = values2(code[i]).x * e[i / 4];
      if (32 * i < n) {
        if constexpr (sizeof(T) == 4)
          to[32 * i] = v;
        else
          to[32 * i] = __float2bfloat16_rn(v);
      }
    }
  }
}

}  // namespace

cudaError_t launch_encode8(const Encode8Params& p, int dtype, int block_rows, int sms, cudaStream_t st) {
  const auto kernel = dtype == XP_F32 ? (block_rows == 1 ? encode_kernel<float, false> : encode_kernel<float, true>)
                                      : (block_rows == 1 ? encode_kernel<bf16, false> : encode_kernel<bf16, true>);
  const size_t smem = sizeof(unsigned) * (128 * 32 + kWarps * 128) + (size_t)128 * 128 * (dtype == XP_F32 ? 4 : 2);
  return launch_dependent(kernel, dim3(p.tiles < 2u * sms ? p.tiles : 2u * sms), kThreads, smem, 1, st, p);
}

template <typename T, unsigned kPiece>
cudaError_t decode(const Decode8Params& p, cudaStream_t st) {
  const u64 pieces = (u64)((p.cols + kPiece - 1) / kPiece) * p.rows, per_cta = kDecodeThreads / 32;
  return launch_dependent(decode_kernel<T, kPiece>, dim3((unsigned)((pieces + per_cta - 1) / per_cta)), kDecodeThreads, 0, 1, st, p);
}

// Short rows leave much of a long piece empty (to bf16, 256 columns a piece and 1024: 60000 x 65 9.7 and 27 us, 12000 x
// 1031 11.7 and 14.0), but where rows are aligned a piece of 256 is one load for a lane (12000 x 1032 11.7 and 9.1).
cudaError_t launch_decode8(const Decode8Params& p, int dtype, cudaStream_t st) {
  const bool aligned = p.aligned && p.cols % (dtype == XP_F32 ? 4 : 8) == 0, few = p.cols <= (aligned ? 256 : 1280);
  if (dtype == XP_F32) return few ? decode<float, 256>(p, st) : decode<float, 1024>(p, st);
  return few ? decode<bf16, 256>(p, st) : decode<bf16, 1024>(p, st);
}

}  // namespace xp
