// Layer norm, forward and backward, with the reduction of the weight's
// gradient over the rows.  include/xp_train.h states the formulas.
//
// Both directions read and write every element once and compute a handful of
// operations on it: HBM bounds them.  A row belongs to a group of threads
// that keeps it on chip between its sums and its output: a warp (short rows),
// a part of a CTA or a whole one, or the CTAs of a thread-block cluster, each
// with a slice of the row (long rows, and rows too few to fill the GPU).
#include "xp_train_device.cuh"

namespace xp {
namespace {

typedef __nv_bfloat16 bf16;
typedef unsigned long long u64;

// who shares a row
enum { kWarp = 0, kCta = 1, kCluster = 2, kHalf = 3 };   // kHalf: half a warp
// A row's threads in one warp, side by side.
template <int MODE>
constexpr int kLanes = MODE == kHalf ? 16 : 32;
constexpr int kMaxWarps = 32;
constexpr int kMaxCluster8 = 8;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }

// ---- units: the V elements (16 bytes) a thread takes at once, as V / 2 pairs.
// In rows that allow it they lie side by side.  In others (NARROW: lengths,
// strides or addresses that are no multiple of 16 bytes) a warp's lanes take
// neighbouring pairs, 64 columns at a time (of fp32 a pair is 32 columns apart),
// so that words at any offset are read and written side by side.
template <typename T>
constexpr int kUnit = 16 / (int)sizeof(T);

template <typename T, bool NARROW>
constexpr int kApart = NARROW && sizeof(T) == 4 ? 32 : 1;   // of a pair's columns

__device__ __forceinline__ float lo_of(unsigned w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(unsigned w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float2 both(float f) { return make_float2(f, f); }

template <typename T, int P>
__device__ __forceinline__ void unpack16(uint4 q, float2 (&f)[P]) {
  if constexpr (sizeof(T) == 4) {
    f[0] = make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
    f[1] = make_float2(__uint_as_float(q.z), __uint_as_float(q.w));
  } else {
    f[0] = make_float2(lo_of(q.x), hi_of(q.x));
    f[1] = make_float2(lo_of(q.y), hi_of(q.y));
    f[2] = make_float2(lo_of(q.z), hi_of(q.z));
    f[3] = make_float2(lo_of(q.w), hi_of(q.w));
  }
}
__device__ __forceinline__ unsigned pack2(float2 f) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const unsigned*>(&h);
}
template <typename T, int P>
__device__ __forceinline__ uint4 pack16(const float2 (&f)[P]) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x), __float_as_uint(f[1].y));
  else
    return make_uint4(pack2(f[0]), pack2(f[1]), pack2(f[2]), pack2(f[3]));
}
// A unit of gamma or beta (w is aligned to 16 bytes); `none` where there is
// none.  No branches: the loads of several units are in flight together.
// (Plain loads, here and of the statistics: a load that may assume read-only
// memory could be moved before the wait for the kernel that writes it.)
// Eight floats are one load of 32 bytes where they are aligned for it: in two of
// 16 a warp takes every other piece of its lines, twice the L1 cycles (16384 x
// 4096 bf16 with fp32 weights: 48.4 us, 57.6 by two loads).
template <typename W, int P>
__device__ __forceinline__ void load_whole_w(const W* p, bool has, float none, float2 (&f)[P]) {
  if constexpr (sizeof(W) == 4 && P == 4) {
    const bool aligned = (reinterpret_cast<uintptr_t>(p) & 31u) == 0;
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = none;
    asm volatile(
        "{\n.reg .pred p, q;\nsetp.ne.u32 p, %9, 0;\nsetp.ne.u32 q, %10, 0;\n"
        "@p ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n"
        "@q ld.global.v4.f32 {%0, %1, %2, %3}, [%8];\n"
        "@q ld.global.v4.f32 {%4, %5, %6, %7}, [%8 + 16];\n}"
        : "+f"(e[0]), "+f"(e[1]), "+f"(e[2]), "+f"(e[3]), "+f"(e[4]), "+f"(e[5]), "+f"(e[6]), "+f"(e[7])
        : "l"(p), "r"((unsigned)(has && aligned)), "r"((unsigned)(has && !aligned))
        : "memory");
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = make_float2(e[2 * i], e[2 * i + 1]);
  } else if constexpr (sizeof(W) == 4) {
    const float4 rest = make_float4(none, none, none, none);
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const float4 q = has ? reinterpret_cast<const float4*>(p)[i] : rest;
      f[2 * i] = make_float2(q.x, q.y);
      f[2 * i + 1] = make_float2(q.z, q.w);
    }
  } else {
    const unsigned rest = pack2(both(none));
    uint4 q = make_uint4(rest, rest, rest, rest);
    if constexpr (P == 4) {
      q = has ? *reinterpret_cast<const uint4*>(p) : q;
    } else {
      const uint2 h = has ? *reinterpret_cast<const uint2*>(p) : make_uint2(rest, rest);
      q.x = h.x, q.y = h.y;
    }
    const unsigned words[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < P; ++i) f[i] = make_float2(lo_of(words[i]), hi_of(words[i]));
  }
}
// A unit of gamma or beta: pair i begins at column c + i * 64 (NARROW) or c + 2 i
// of the slice, which begins at column c0 and has `cols`.  `whole`, the same
// for a warp: every lane's unit lies in the slice.
template <typename T, typename W, bool NARROW, int P>
__device__ __forceinline__ void load_w(const void* w, unsigned c0, int c, int cols, bool whole, float none, float2 (&f)[P]) {
  const W* p = static_cast<const W*>(w) + c0 + c;
  if constexpr (!NARROW) {
    load_whole_w<W, P>(p, w && c < cols, none, f);
  } else if (sizeof(T) == 2 && whole && w && (reinterpret_cast<uintptr_t>(w) & (2 * sizeof(W) - 1)) == 0) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if constexpr (sizeof(W) == 4) {
        f[i] = *reinterpret_cast<const float2*>(p + 64 * i);
      } else {
        const unsigned q = *reinterpret_cast<const unsigned*>(p + 64 * i);
        f[i] = make_float2(lo_of(q), hi_of(q));
      }
    }
  } else {
    constexpr int kNext = kApart<T, NARROW>;
    const int n = w ? cols - c : 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      f[i].x = 64 * i < n ? to_f(p[64 * i]) : none;
      f[i].y = 64 * i + kNext < n ? to_f(p[64 * i + kNext]) : none;
    }
  }
}

// ---- sums over the threads of a row
__device__ __forceinline__ void group_bar(int group, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
}
__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_size() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void store_remote(const float* p, unsigned rank, float v) {
  unsigned a = (unsigned)__cvta_generic_to_shared(p), r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(r), "f"(v) : "memory");
}

__host__ __device__ constexpr int log2_of(int n) { return n <= 1 ? 0 : 1 + log2_of(n / 2); }

// N sums at once (a power of two): at each step a lane keeps half of its
// values and hands the other half to its partner, so N of them cost
// N - 1 + 5 - log2 N shuffles and not 5 N.  Lane l ends with the warp's sum of
// value l >> (5 - log2 N).
template <int N, int LANES>
__device__ __forceinline__ float warp_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int o = LANES / 2;
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2, o /= 2) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float keep = upper ? v[n + i] : v[i], give = upper ? v[i] : v[n + i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
#pragma unroll
  for (; o > 0; o /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

// Shared words of N sums.  Two buffers in turn: a thread that reads one meets
// the others at the next sums' barrier before it is written again.
template <int N>
struct SumWords {
  float warp[2][kMaxWarps][N];
  float cta[2][kMaxCluster8][N];
};

// N values summed over the row's threads: value i of the result is in lane i
// (and i + N, ...) of every warp.  Each warp's sums, the group meets, the
// warps' sums added up; in a cluster the same once more among its CTAs,
// through their shared memory.  The order of the additions is fixed.
template <int MODE, int N>
__device__ __forceinline__ float row_sums(float (&v)[N], SumWords<N>& w, int buf, int group, int threads) {
  constexpr int L = log2_of(N);
  const int lane = threadIdx.x & 31;
  float t = warp_sums<N, kLanes<MODE>>(v);
  if constexpr (MODE == kWarp || MODE == kHalf)
    return __shfl_sync(0xffffffffu, t, (lane & (N - 1)) << (log2_of(kLanes<MODE>) - L), kLanes<MODE>);
  if ((lane & ((32 >> L) - 1)) == 0) w.warp[buf][threadIdx.x >> 5][lane >> (5 - L)] = t;
  if constexpr (MODE == kCluster)
    __syncthreads();
  else
    group_bar(group, threads);
  const int nw = threads >> 5, first = group * nw;
  t = 0.f;
  for (int j = lane >> L; j < nw; j += 32 >> L) t += w.warp[buf][first + j][lane & (N - 1)];
#pragma unroll
  for (int o = N; o < 32; o *= 2) t += __shfl_xor_sync(0xffffffffu, t, o);
  if constexpr (MODE == kCluster) {
    const unsigned n = cluster_size();
    if (threadIdx.x < N * n) store_remote(&w.cta[buf][cluster_rank()][lane & (N - 1)], threadIdx.x >> L, t);
    cluster_arrive();
    cluster_wait();
    t = 0.f;
    for (unsigned r = 0; r < n; ++r) t += w.cta[buf][r][lane & (N - 1)];
  }
  return t;
}

// ---- rows on their way from global to shared memory
__device__ __forceinline__ void copy_async16(unsigned smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}
// the first `bytes` bytes, zeros after
__device__ __forceinline__ void copy_async16(unsigned smem, const void* gmem, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(bytes) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the newest n groups of this thread's copies have landed
__device__ __forceinline__ void wait_groups(int n) {
  if (n == 0)
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 1;" ::: "memory");
}
// One turn's rows are in work, the next ones' on their way.  (More would be
// filled before the first turn: 60000 x 304 bf16 31.9 us, 33.1 with up to 8.)
constexpr int kMaxStages = 2;

// A row (one CTA's slice of it) in shared memory: each warp's 32 NV units side
// by side, and one more where a row may begin within one.
template <typename T, bool NARROW, int NV>
constexpr unsigned kWarpBytes = 32 * NV * 16 + (NARROW ? 16 : 0);
template <typename T, bool NARROW, int NV>
__host__ __device__ constexpr unsigned row_bytes(unsigned threads) {
  return threads == 16 ? 16 * NV * 16 : (threads >> 5) * kWarpBytes<T, NARROW, NV>;
}

// How a row of a matrix gets there: every warp copies the units it will use
// itself.  Thread t's unit k is unit first_unit(t) + 32 k of the row, so the
// distance between a thread's units is the same for every row length.  Past a
// row's end there are zeros, where no copy ever writes.
//
// NARROW: the 16-byte pieces of memory that hold the warp's columns, from the
// one on which its first lies, and zeros from the row's end to the end of the
// units that are read.  The bytes of the first piece before the row are copied
// and not used; the matrix's first row has none.
// (kHalf: LANES = 16, and the half's units for the warp's.)
template <int NV>
__device__ __forceinline__ int first_unit(int tid) {
  return (tid & ~31) * NV + (tid & 31);
}
// The first column of a thread's pair i of unit k.
template <typename T, bool NARROW, int E, int LANES = 32>
__device__ __forceinline__ int column(int tid, int k, int i) {
  constexpr int V = kUnit<T>;
  if (!NARROW) return (first_unit<E / V>(tid) + LANES * k) * V + 2 * i;
  return (tid & ~31) * E + (k * V / 2 + i) * 64 + (tid & 31) * (sizeof(T) == 2 ? 2 : 1);
}

template <typename T, bool NARROW, int NV, int LANES = 32>
__device__ __forceinline__ void fetch_row(const T* row, int cols, const T* matrix, unsigned smem, int tid) {
  const int lane = tid & 31;
  if constexpr (!NARROW) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (first_unit<NV>(tid) + LANES * k) * kUnit<T>;
      if (c < cols) copy_async16(smem + (lane + LANES * k) * 16, row + c);
    }
  } else {
    const int shift = (int)(reinterpret_cast<uintptr_t>(row) & 15u), first = (tid & ~31) * NV * 16;
    const char* from = reinterpret_cast<const char*>(row) - shift + first;
    const int bytes = shift + cols * (int)sizeof(T) - first;   // of the row, from there
    if (bytes <= shift) return;
    const bool before = from < reinterpret_cast<const char*>(matrix);
    if (bytes >= 32 * NV * 16 + 16 && !before) {
#pragma unroll
      for (int k = 0; k < NV; ++k) copy_async16(smem + (lane + 32 * k) * 16, from + (lane + 32 * k) * 16);
      if (lane == 0) copy_async16(smem + 32 * NV * 16, from + 32 * NV * 16);
      return;
    }
#pragma unroll
    for (int k = 0; k <= NV; ++k) {
      const int at = (lane + 32 * k) * 16;
      // a unit that is read, or the piece behind the last of them
      if (k == NV || 32 * k * 16 >= bytes - shift) {
        if (lane == 0) copy_async16(smem + at, from + min(at, (bytes - 1) & ~15), min(max(bytes - at, 0), 16));
        break;
      }
      if (k > 0 || lane > 0 || !before) copy_async16(smem + at, from + min(at, (bytes - 1) & ~15), min(max(bytes - at, 0), 16));
    }
    if (lane == 0 && before) {
      for (int j = 0; j < 16 / (int)sizeof(T); ++j) {
        const int c = j - shift / (int)sizeof(T);
        if constexpr (sizeof(T) == 4)
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(smem + 4 * j), "r"(c >= 0 && c < cols ? reinterpret_cast<const unsigned*>(row)[c] : 0u) : "memory");
        else
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(smem + 2 * j), "h"(c >= 0 && c < cols ? reinterpret_cast<const unsigned short*>(row)[c] : (unsigned short)0) : "memory");
      }
    }
  }
}

// Loads from shared memory by its 32-bit address.  (Volatile: they stay behind
// the wait for the copies.)
__device__ __forceinline__ uint4 load_shared16(unsigned a) {
  uint4 q;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(a));
  return q;
}
__device__ __forceinline__ unsigned load_shared4(unsigned a) {
  unsigned w;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(a));
  return w;
}

// A row in shared memory, as a warp reads it.
template <typename T, bool NARROW, int LANES = 32>
struct Landed {
  unsigned at;       // the lane's unit, or (NARROW) the word with its first column
  unsigned select;   // which halves of two words are a pair

  __device__ __forceinline__ Landed(unsigned smem, const T* row, int lane) {
    const unsigned shift = (unsigned)(reinterpret_cast<uintptr_t>(row) & 15u);
    at = NARROW ? smem + (shift & ~3u) + 4 * lane : smem + 16 * lane;
    select = shift & 2u ? 0x5432u : 0x3210u;
  }
  // the lane's unit k
  __device__ __forceinline__ uint4 raw(int k) const {
    if constexpr (!NARROW) {
      return load_shared16(at + 16 * LANES * k);
    } else {
      unsigned w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = load_shared4(at + 512 * k + 128 * i);
      if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __byte_perm(w[i], load_shared4(at + 512 * k + 128 * i + 4), select);
      }
      return make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ void read(int k, float2 (&f)[kUnit<T> / 2]) const { unpack16<T, kUnit<T> / 2>(raw(k), f); }
};

// Clears what no copy will ever write (not NARROW).
template <typename T, int NV, int LANES>
__device__ __forceinline__ void clear_rows(unsigned smem, unsigned row_len, int nrows, int cols, int tid) {
  const int lane = tid & 31;
  for (int r = 0; r < nrows; ++r, smem += row_len) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if ((first_unit<NV>(tid) + LANES * k) * kUnit<T> >= cols)
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(smem + (lane + LANES * k) * 16), "r"(0) : "memory");
    }
  }
}

// A warp's part of an output row (NARROW), unit by unit in their order, in
// words: where they begin at odd columns, a lane's word has the second half
// of the pair before its own.  n columns are left at the warp's first, `out`.
template <typename T, int E>
struct Written {
  T* out;
  int n, lane;
  unsigned last;   // lane 0: the last lane's pair of the 64 columns before

  __device__ __forceinline__ Written(T* row, int cols, int tid) : out(row + (tid & ~31) * E), n(cols - (tid & ~31) * E), lane(tid & 31), last(0) {}
  __device__ __forceinline__ void put(int k, const float2 (&f)[kUnit<T> / 2]) {
    if (32 * kUnit<T> * (k + 1) <= n)
      put_unit<true>(k, f);
    else
      put_unit<false>(k, f);
  }
  template <bool whole>
  __device__ __forceinline__ void put_unit(int k, const float2 (&f)[kUnit<T> / 2]) {
    constexpr int P = kUnit<T> / 2;
    const int at = 64 * P * k;
    if constexpr (sizeof(T) == 4) {
      float* o = out + at + lane;
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (whole || at + 64 * i + lane < n) o[64 * i] = f[i].x;
        if (whole || at + 64 * i + 32 + lane < n) o[64 * i + 32] = f[i].y;
      }
    } else {
      unsigned short* o = reinterpret_cast<unsigned short*>(out) + at + 2 * lane;
      const int mine = n - at - 2 * lane;   // columns from this lane's first on
      if ((reinterpret_cast<uintptr_t>(out) & 2u) == 0) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const unsigned w = pack2(f[i]);
          if (whole || 64 * i + 1 < mine)
            *reinterpret_cast<unsigned*>(o + 64 * i) = w;
          else if (64 * i < mine)
            o[64 * i] = (unsigned short)w;
        }
      } else {
        unsigned w = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          w = pack2(f[i]);
          const unsigned left = __shfl_sync(0xffffffffu, w, (lane + 31) & 31);
          const unsigned word = __byte_perm(lane ? left : last, w, 0x5432);
          last = left;
          if (i == 0 && k == 0 && lane == 0) {
            if (whole || n > 0) o[0] = (unsigned short)w;
          } else if (whole || 64 * i < mine) {
            *reinterpret_cast<unsigned*>(o + 64 * i - 1) = word;
          }
          if (!whole && 64 * i + 2 == mine) o[64 * i + 1] = (unsigned short)(w >> 16);   // the row's last column
        }
        // the warp's last column, or the row's
        if (whole && lane == 31 && (k == E / (2 * P) - 1 || at + 64 * P == n)) o[64 * P - 63] = (unsigned short)(w >> 16);
      }
    }
  }
};

// ---------------------------------------------------------------- forward

// One row per group, in registers from its load to its output: E elements per
// thread.  The CTAs are small and many: eight of 128 threads are on an SM, so
// that one's sums are another's loads, and the hardware hands the rows out.
//   Measured at 16384 x 4096 bf16 (268 MB, a plain copy of it takes 42 us):
//   32 elements per thread 45 us, 6.0 TB/s; 16 elements 49, 8 elements 68; one
//   persistent CTA per SM with a warp per row and rows copied ahead 50.
// R > 1: rows side by side, in rows of 256 columns and fewer, so that a warp
// has more in flight (60000 x 96 bf16: 9 us, 16 with one row).  Up to 128 columns
// a row is half a warp's, or half of the lanes would have none (6.4 us; 200000 x
// 64: 14, 25 with whole warps).
constexpr int kForwardThreads = 1024;   // of an SM at least
template <typename T, bool NARROW, int E, int R, int MODE, int MAXT>
__global__ void __launch_bounds__(MAXT, kForwardThreads / MAXT) ln_forward_kernel(const __grid_constant__ NormRowsParams prm) {
  extern __shared__ uint4 s_dyn[];
  __shared__ SumWords<R> words;
  constexpr int V = kUnit<T>, NV = E / V, P = V / 2;
  constexpr int L = kLanes<MODE>;
  constexpr bool kRows = MODE == kWarp || MODE == kHalf;   // a CTA has several
  const int threads = kRows ? L : blockDim.x;
  const int tid = kRows ? threadIdx.x & (L - 1) : threadIdx.x, u0 = first_unit<NV>(tid), lane = threadIdx.x & 31;
  const int w0 = (tid & ~31) * E;   // the warp's first column
  constexpr bool kSkip = NARROW || E > 32;
  const unsigned csize = MODE == kCluster ? cluster_size() : 1;
  const u64 row = R * (kRows ? (u64)blockIdx.x * (blockDim.x / L) + threadIdx.x / L : blockIdx.x / csize);
  const unsigned c0 = MODE == kCluster ? cluster_rank() * E * threads : 0;
  const int cols = c0 < prm.cols ? (int)min((unsigned)E * threads, prm.cols - c0) : 0;   // a cluster's last CTA may have none
  const int left = (int)min(prm.rows - min(row, prm.rows), (u64)R);
  const T* x = static_cast<const T*>(prm.x) + row * prm.x_stride + c0;
  constexpr unsigned kRow = kWarpBytes<T, NARROW, NV>;
  const unsigned slot = (unsigned)__cvta_generic_to_shared(s_dyn) + (threadIdx.x >> 5) * R * kRow;   // [warp][r]
  if (MODE == kCluster) cluster_arrive();   // its end: every CTA of the cluster runs
  wait_for_predecessors();
  let_successor_start();
  if (MODE == kWarp && left == 0) return;

  uint4 q[R][NV];   // as they came: bf16 take half the registers their values would
  if constexpr (!NARROW) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint4* a = reinterpret_cast<const uint4*>(x + r * prm.x_stride);
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const int u = u0 + L * k;
        q[r][k] = r < left && u * V < cols ? __ldcs(a + u) : make_uint4(0, 0, 0, 0);
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (r < left) fetch_row<T, NARROW, NV>(x + r * prm.x_stride, cols, static_cast<const T*>(prm.x), slot + r * kRow, tid);
    commit();
    wait_groups(0);
    __syncwarp();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const Landed<T, NARROW> here(slot + r * kRow, x + r * prm.x_stride, lane);
#pragma unroll
      for (int k = 0; k < NV; ++k) q[r][k] = r < left && w0 + 32 * k * V < cols ? here.raw(k) : make_uint4(0, 0, 0, 0);
    }
  }
  float v[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (kSkip && w0 + 32 * k * V >= cols) break;   // nothing there for this warp
      float2 f[P];
      unpack16<T, P>(q[r][k], f);
#pragma unroll
      for (int i = 0; i < P; ++i) sum = __fadd2_rn(sum, f[i]);
    }
    v[r] = sum.x + sum.y;
  }
  if (MODE == kCluster) cluster_wait();
  const float inv = 1.0f / (float)prm.cols;
  const float means = row_sums<MODE, R>(v, words, 0, 0, threads) * inv;   // row r's in lane r
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float mean = R > 1 ? __shfl_sync(0xffffffffu, means, r, L) : means;
    float2 sq = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      if (kSkip && w0 + 32 * k * V >= cols) break;
      float2 f[P];
      unpack16<T, P>(q[r][k], f);
      if (NARROW && w0 + 32 * (k + 1) * V > cols) {
        const int n = cols - column<T, NARROW, E>(tid, k, 0);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float2 d = __fadd2_rn(f[i], make_float2(n > 64 * i ? -mean : 0.f, n > 64 * i + kApart<T, NARROW> ? -mean : 0.f));
          sq = __ffma2_rn(d, d, sq);
        }
      } else {
        const float2 m = both(NARROW || (u0 + L * k) * V < cols ? -mean : 0.f);   // a unit is whole or absent
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float2 d = __fadd2_rn(f[i], m);
          sq = __ffma2_rn(d, d, sq);
        }
      }
    }
    v[r] = sq.x + sq.y;
  }
  const float rstds = 1.0f / sqrtf(row_sums<MODE, R>(v, words, 1, 0, threads) * inv + prm.eps);
  if (tid < left && c0 == 0) {
    if (prm.mean) prm.mean[row + tid] = means;
    if (prm.rstd) prm.rstd[row + tid] = rstds;
  }
  T* y = static_cast<T*>(prm.out) + row * prm.out_stride + c0;
  auto output = [&](auto w) {
    typedef decltype(w) W;
    [[maybe_unused]] unsigned last[R] = {};
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = column<T, NARROW, E, L>(tid, k, 0);
      if (kSkip && w0 + 32 * k * V >= cols) break;
      const bool whole = w0 + 32 * (k + 1) * V <= cols;
      float2 g[P], b[P];
      load_w<T, W, NARROW, P>(prm.gamma, c0, c, cols, whole, 1.f, g);
      load_w<T, W, NARROW, P>(prm.beta, c0, c, cols, whole, 0.f, b);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float2 mean = both(-(R > 1 ? __shfl_sync(0xffffffffu, means, r, L) : means)), rstd = both(R > 1 ? __shfl_sync(0xffffffffu, rstds, r, L) : rstds);
        float2 o[P];
        unpack16<T, P>(q[r][k], o);
#pragma unroll
        for (int i = 0; i < P; ++i) o[i] = __ffma2_rn(__fmul2_rn(__fadd2_rn(o[i], mean), rstd), g[i], b[i]);
        if constexpr (NARROW) {
          Written<T, E> to(y + r * prm.out_stride, r < left ? cols : 0, tid);
          to.last = last[r];
          to.put(k, o);
          last[r] = to.last;
        } else {
          if (r < left && c < cols) *reinterpret_cast<uint4*>(y + r * prm.out_stride + c) = pack16<T, P>(o);
        }
      }
    }
  };
  if (prm.gamma_bf16)
    output(bf16());
  else
    output(float());
}

// ---------------------------------------------------------------- backward

// Each group walks over the rows, R at a time, and keeps its columns' sums of
// dgamma and dbeta in registers: a grid of no more CTAs than the GPU holds, so
// that few partial sums are left.  Asynchronous copies bring the next R rows
// into shared memory; a row is read from there twice, for its sums and for
// dx: with d = x - mean and a = dy * gamma,
//   dx = rstd (a - sum(a) / cols - d rstd (rstd sum(a d) / cols)),
// dgamma += (dy rstd) d, dbeta += dy.  (No power of rstd is formed: its cube
// leaves fp32's range for rows beyond 1e13 and below 1e-13, while sum(a d)
// rstd and d rstd are of the size of a and 1.)  R rows share a barrier, and
// their sums' latencies overlap.
template <typename T, bool NARROW, int E, int R, int MODE>
__global__ void __launch_bounds__(512, 1) ln_backward_kernel(const __grid_constant__ NormRowsParams prm) {
  extern __shared__ uint4 s_dyn[];
  __shared__ SumWords<2 * R> words;
  constexpr int V = kUnit<T>, NV = E / V, P = V / 2;
  constexpr bool kKeepGamma = E <= 16;                   // else in shared memory, a unit per thread as the rows'
  constexpr int L = kLanes<MODE>;
  const int threads = MODE == kWarp || MODE == kHalf ? L : prm.threads;
  const int group = MODE == kCluster ? 0 : threadIdx.x / threads;
  const int tid = threadIdx.x - group * threads, u0 = first_unit<NV>(tid), lane = threadIdx.x & (L - 1);
  const int groups = MODE == kCluster ? 1 : blockDim.x / threads;
  const unsigned csize = MODE == kCluster ? cluster_size() : 1;
  const unsigned part = blockIdx.x / csize;
  const unsigned width = E * threads;                    // columns of a CTA
  const unsigned c0 = MODE == kCluster ? cluster_rank() * width : 0;
  const int cols = c0 < prm.cols ? (int)min(width, prm.cols - c0) : 0;   // a cluster's last CTA may have none
  const float inv = 1.0f / (float)prm.cols;
  const int stages = prm.stages;
  // shared memory: [group][stage][r][x, dy][warp], then gamma
  const unsigned len = row_bytes<T, NARROW, NV>(threads);
  const unsigned slot = (unsigned)__cvta_generic_to_shared(s_dyn) + group * stages * R * 2 * len + (tid >> 5) * kWarpBytes<T, NARROW, NV>;
  const int rows = (int)prm.rows, step = (int)prm.nparts * groups * R;
  const int first = ((int)part * groups + group) * R;
  if constexpr (!NARROW) clear_rows<T, NV, L>(slot, len, stages * R * 2, cols, tid);
  wait_for_predecessors();

  // The row in work; what a turn is further in each matrix.
  const T* x = static_cast<const T*>(prm.x) + (u64)first * prm.x_stride + c0;
  const T* dy = static_cast<const T*>(prm.dy) + (u64)first * prm.dy_stride + c0;
  T* dx = static_cast<T*>(prm.out) + (u64)first * prm.out_stride + c0;
  const u64 x_turn = step * prm.x_stride, dy_turn = step * prm.dy_stride;
  // `left` rows from a turn's first one on, to stage `to`
  auto fetch_rows = [&](const T* fx, const T* fd, int left, int to) {
    unsigned at = slot + to * R * 2 * len;
#pragma unroll
    for (int r = 0; r < R; ++r, at += 2 * len, fx += prm.x_stride, fd += prm.dy_stride) {
      if (r < left) {
        fetch_row<T, NARROW, NV, L>(fx, cols, static_cast<const T*>(prm.x), at, tid);
        fetch_row<T, NARROW, NV, L>(fd, cols, static_cast<const T*>(prm.dy), at + len, tid);
      }
    }
    commit();
  };
  for (int s = 0; s < stages; ++s) fetch_rows(x + s * x_turn, dy + s * dy_turn, rows - first - s * step, s);

  float2 dg[NV][P], db[NV][P];
  float2 gam[kKeepGamma ? NV : 1][P];
  float* s_gam = reinterpret_cast<float*>(reinterpret_cast<char*>(s_dyn) + (size_t)groups * stages * R * 2 * len) + group * width;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = column<T, NARROW, E, L>(tid, k, 0);
    float2 w[P];
    if (prm.gamma_bf16)
      load_w<T, bf16, NARROW, P>(prm.gamma, c0, c, cols, false, 1.f, w);
    else
      load_w<T, float, NARROW, P>(prm.gamma, c0, c, cols, false, 1.f, w);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      dg[k][i] = db[k][i] = make_float2(0.f, 0.f);
      if constexpr (kKeepGamma)
        gam[k][i] = w[i];
      else
        reinterpret_cast<float2*>(s_gam + (u0 + L * k) * V)[i] = w[i];   // read back by this thread alone
    }
  }
  auto gammas = [&](int k, float2 (&w)[P]) {
    if constexpr (kKeepGamma) {
#pragma unroll
      for (int i = 0; i < P; ++i) w[i] = gam[k][i];
    } else {
      const float* p = s_gam + (u0 + L * k) * V;
#pragma unroll
      for (int i = 0; i < P; i += 2) {
        const float4 q = reinterpret_cast<const float4*>(p)[i / 2];
        w[i] = make_float2(q.x, q.y);
        w[i + 1] = make_float2(q.z, q.w);
      }
    }
  };
  // lane r of each warp holds the statistics of the turn's row r
  float mean_next = 0.f, rstd_next = 0.f;
  auto statistics = [&](int row) {
    if (lane < R && row + lane < rows) {
      mean_next = prm.mean[row + lane];
      rstd_next = prm.rstd[row + lane];
    }
  };
  statistics(first);
  if (MODE == kCluster) {   // every CTA of the cluster runs before its shared memory is written
    cluster_arrive();
    cluster_wait();
  }
  int stage = 0, buf = 0;
  const int behind = MODE == kHalf ? (group & 1) * R : 0;   // the halves of a warp end their loops together
  for (int row = first; row - behind < rows; row += step, x += x_turn, dy += dy_turn, dx += step * prm.out_stride) {
    const float means = mean_next, rstds = rstd_next;
    const int left = rows - row;
    statistics(row + step);
    wait_groups(stages - 1);
    if constexpr (NARROW) __syncwarp();   // the other lanes' copies have landed too
    const unsigned here = slot + stage * R * 2 * len;
    float v[2 * R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      float2 sa = make_float2(0.f, 0.f), sd = sa;
      const float2 mean = both(-__shfl_sync(0xffffffffu, means, r, L)), rstd = both(__shfl_sync(0xffffffffu, rstds, r, L));
      if (r < left) {
        const Landed<T, NARROW, L> hx(here + r * 2 * len, x + r * prm.x_stride, lane), hd(here + (r * 2 + 1) * len, dy + r * prm.dy_stride, lane);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          if (NARROW && (u0 - lane + 32 * k) * V >= cols) continue;   // nothing there for this warp
          float2 fx[P], fd[P], w[P];
          hx.read(k, fx);
          hd.read(k, fd);
          gammas(k, w);
#pragma unroll
          for (int i = 0; i < P; ++i) {   // dy is 0 past the row's end
            const float2 d = __fadd2_rn(fx[i], mean), a = __fmul2_rn(fd[i], w[i]);
            sa = __fadd2_rn(sa, a);
            sd = __ffma2_rn(a, d, sd);
            dg[k][i] = __ffma2_rn(__fmul2_rn(fd[i], rstd), d, dg[k][i]);
            db[k][i] = __fadd2_rn(db[k][i], fd[i]);
          }
        }
      }
      v[2 * r] = sa.x + sa.y;
      v[2 * r + 1] = sd.x + sd.y;
    }
    const float sums = row_sums<MODE, 2 * R>(v, words, buf, group, threads) * inv;
    buf ^= 1;
    T* out = dx;
#pragma unroll
    for (int r = 0; r < R; ++r, out += prm.out_stride) {
      const float mean = __shfl_sync(0xffffffffu, means, r, L), rstd = __shfl_sync(0xffffffffu, rstds, r, L);
      const float sum_a = __shfl_sync(0xffffffffu, sums, 2 * r, L), sum_ad = __shfl_sync(0xffffffffu, sums, 2 * r + 1, L);
      if (r < left) {
        const Landed<T, NARROW, L> hx(here + r * 2 * len, x + r * prm.x_stride, lane), hd(here + (r * 2 + 1) * len, dy + r * prm.dy_stride, lane);
        const float2 k1 = both(-sum_a), k2 = both(-(rstd * sum_ad) * rstd);
        Written<T, E> to(out, cols, tid);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          if (NARROW && (u0 - lane + 32 * k) * V >= cols) continue;
          float2 fx[P], fd[P], w[P];
          hx.read(k, fx);
          hd.read(k, fd);
          gammas(k, w);
#pragma unroll
          for (int i = 0; i < P; ++i)
            fd[i] = __fmul2_rn(__ffma2_rn(__fadd2_rn(fx[i], both(-mean)), k2, __ffma2_rn(fd[i], w[i], k1)), both(rstd));
          const int c = (u0 + L * k) * V;
          if constexpr (NARROW) {
            to.put(k, fd);
          } else {
            if (c < cols) *reinterpret_cast<uint4*>(out + c) = pack16<T, P>(fd);
          }
        }
      }
    }
    if constexpr (NARROW) __syncwarp();   // every lane has read these rows
    fetch_rows(x + stages * x_turn, dy + stages * dy_turn, left - stages * step, stage);
    if (++stage == stages) stage = 0;
  }
  wait_groups(0);
  let_successor_start();
  if (!prm.dgamma) return;

  // the groups' sums, added in their order, then one part of the CTA or cluster
  float* out_g = (prm.nparts > 1 ? prm.partial + (size_t)part * 2 * prm.cols : prm.dgamma) + c0;
  float* out_b = (prm.nparts > 1 ? prm.partial + ((size_t)part * 2 + 1) * prm.cols : prm.dbeta) + c0;
  const bool add = prm.nparts == 1 && prm.accumulate;
  if constexpr (MODE == kHalf) {   // a warp's two groups first: the sums of the lower one
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        dg[k][i].x += __shfl_down_sync(0xffffffffu, dg[k][i].x, 16);
        dg[k][i].y += __shfl_down_sync(0xffffffffu, dg[k][i].y, 16);
        db[k][i].x += __shfl_down_sync(0xffffffffu, db[k][i].x, 16);
        db[k][i].y += __shfl_down_sync(0xffffffffu, db[k][i].y, 16);
      }
    }
  }
  if (groups > 1) {
    float* acc = reinterpret_cast<float*>(s_dyn);   // [2][width]
    for (int g = 0; g < groups; g += 32 / L) {
      __syncthreads();
      if (g != group) continue;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          float* a = acc + column<T, NARROW, E, L>(tid, k, i);
          float* b = a + width;
          if constexpr (kApart<T, NARROW> == 1) {
            float2* a2 = reinterpret_cast<float2*>(a);
            float2* b2 = reinterpret_cast<float2*>(b);
            *a2 = g ? __fadd2_rn(*a2, dg[k][i]) : dg[k][i];
            *b2 = g ? __fadd2_rn(*b2, db[k][i]) : db[k][i];
          } else {
            a[0] = g ? a[0] + dg[k][i].x : dg[k][i].x;
            a[32] = g ? a[32] + dg[k][i].y : dg[k][i].y;
            b[0] = g ? b[0] + db[k][i].x : db[k][i].x;
            b[32] = g ? b[32] + db[k][i].y : db[k][i].y;
          }
        }
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += blockDim.x) {
      out_g[c] = add ? out_g[c] + acc[c] : acc[c];
      out_b[c] = add ? out_b[c] + acc[width + c] : acc[width + c];
    }
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (u0 + L * k) * V;
      if (!NARROW && !add && prm.nparts > 1) {   // the parts' rows are aligned as the units are
        if (c < cols) {
#pragma unroll
          for (int i = 0; i < P; i += 2) {
            reinterpret_cast<float4*>(out_g + c)[i / 2] = make_float4(dg[k][i].x, dg[k][i].y, dg[k][i + 1].x, dg[k][i + 1].y);
            reinterpret_cast<float4*>(out_b + c)[i / 2] = make_float4(db[k][i].x, db[k][i].y, db[k][i + 1].x, db[k][i + 1].y);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int at = column<T, NARROW, E, L>(tid, k, i / 2) + (i & 1) * kApart<T, NARROW>;
          if (at < cols) {
            const float vg = i & 1 ? dg[k][i / 2].y : dg[k][i / 2].x, vb = i & 1 ? db[k][i / 2].y : db[k][i / 2].x;
            out_g[at] = add ? out_g[at] + vg : vg;
            out_b[at] = add ? out_b[at] + vb : vb;
          }
        }
      }
    }
  }
}

// The parts' sums, column by column: a lane has C columns (4 where the rows are
// aligned for it), the warps of a CTA every kPartWarps-th part each in two
// chains, then the warps' sums in order.  fp32: the depth is 152 / 32 + 2 + 16
// additions, and fp64 runs at 2 additions per clock and SM here (304 parts of
// 5120 columns took 22 us by it).
constexpr int kPartWarps = 16;
template <int C>
__global__ void __launch_bounds__(32 * kPartWarps) ln_parts_kernel(const float* partial, unsigned nparts, unsigned cols,
                                                                  float* dgamma, float* dbeta, int accumulate) {
  __shared__ float s[kPartWarps][32][C];
  wait_for_predecessors();
  let_successor_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned c = (blockIdx.x * 32 + lane) * C;
  const float* p = partial + (size_t)blockIdx.y * cols + c;
  const size_t stride = (size_t)2 * cols;
  float sum[2][C] = {};
  if (c < cols) {
    for (unsigned k = warp; k < nparts; k += 2 * kPartWarps) {
      float a[2][C] = {};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (k + i * kPartWarps < nparts) {
          const float* q = p + (k + i * kPartWarps) * stride;
          if constexpr (C == 4) {
            const float4 f = *reinterpret_cast<const float4*>(q);
            a[i][0] = f.x, a[i][1] = f.y, a[i][2] = f.z, a[i][3] = f.w;
          } else {
            a[i][0] = *q;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int j = 0; j < C; ++j) sum[i][j] += a[i][j];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < C; ++j) s[warp][lane][j] = sum[0][j] + sum[1][j];
  __syncthreads();
  if (threadIdx.x < 32 * C) {
    const int l = threadIdx.x / C, j = threadIdx.x % C;
    const unsigned at = (blockIdx.x * 32 + l) * C + j;
    if (at < cols) {
      float total = s[0][l][j];
#pragma unroll
      for (int w = 1; w < kPartWarps; ++w) total += s[w][l][j];
      float* out = (blockIdx.y ? dbeta : dgamma) + at;
      *out = accumulate ? *out + total : total;
    }
  }
}

// ---------------------------------------------------------------- launches

int sm_count() {
  static PerDevice known;
  return known.get([](int dev) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      n = 152;
    }
    return n;
  });
}

size_t div_up(size_t a, size_t b) { return (a + b - 1) / b; }
int threads_for(size_t elems, int e) { return elems ? 32 * (int)div_up(elems, (size_t)32 * e) : 32; }

// A row's CTAs: enough that a slice has `most` columns at most, and more where
// the rows are too few for the GPU's SMs, as long as a slice keeps 2048.
int cluster_for(size_t rows, size_t cols, size_t most, size_t sms) {
  int c = (int)div_up(cols, most);
  if (c > kMaxCluster8) c = kMaxCluster8;
  while (2 * c <= kMaxCluster8 && rows * c < sms && cols / (2 * c) >= 2048) c *= 2;
  return c;
}

// Rows in flight per group: as many as `budget` bytes of a CTA's shared memory
// hold, no more than there are turns.
int stages_for(size_t budget, size_t per_stage, u64 turns) {
  u64 n = budget / per_stage;
  if (n > (u64)kMaxStages) n = kMaxStages;
  if (n > turns) n = turns;
  return n < 1 ? 1 : (int)n;
}

constexpr size_t kSmemSm = kMaxDynamicSmem;   // of an SM, less what CTAs take statically
static_assert(sizeof(SumWords<8>) <= kMaxStaticSmem, "a backward CTA's static shared memory");

template <typename T, bool NARROW, int E, int R, int MODE, int MAXT>
cudaError_t forward_e(NormRowsParams& p, int threads, int csize, cudaStream_t st) {
  const int groups = MODE == kWarp || MODE == kHalf ? MAXT / threads : 1;
  const size_t smem = NARROW ? (size_t)R * row_bytes<T, NARROW, E / kUnit<T>>(groups * threads) : 0;
  return launch_dependent(ln_forward_kernel<T, NARROW, E, R, MODE, MAXT>, dim3((unsigned)(div_up(p.rows, (size_t)groups * R) * csize)),
                          groups * threads, smem, csize, st, p);
}

// A thread takes 32 elements, which keeps a CTA small; with rows too few to
// fill the GPU it takes 8, and more threads share a row.  bf16 take half the
// registers, so a thread may have 64: in rows up to 1792 columns, which then
// are one warp's (40000 x 1704: 45 us, 49 with two warps of 32; 30000 x 2016: 42 and
// 41), and beyond 4096, where fewer warps hold the SM's place for a row (12000 columns:
// 50 us, 63 with 32; 8192: 45 and 46; 4000 x 20000: 58 and 90; 4096 itself 46.5
// and 45) unless the rows are few (310 x 8193: 8.5 us, 6.8 with 32).  40 where that makes
// two or four full warps of what were three or five (30000 x 2400: 50 us, 56 with 32;
// against 64: 3000 x 5120 13.2 and 14.5, 13000 x 5120 44.5 and 45.5, 13000 x 4609 unaligned 56 and 61).  Warps of 40 and 64 skip the units of which
// they have no column (60000 x 1056: 46 us, 54 without); with 32 that cost more
// than it gave (8000 x 8160: 48 us, 46 without).  2000 x 40032 takes 86 us (125
// in a cluster of 3).
//   Rows in NARROW's layout: 60000 x 1031 71 us (aligned 1056: 46; 107 when the row
// moved in 4-byte words and was units in shared memory), 20046 x 3877 75.
template <typename T, bool NARROW>
cudaError_t forward(NormRowsParams& p, cudaStream_t st) {
  const size_t sms = sm_count();
  if constexpr (!NARROW) {
    if (p.cols <= 128 && p.rows >= 64 * sms) return forward_e<T, NARROW, 8, 4, kHalf, 128>(p, 16, 1, st);
  }
  if (p.cols <= 256) {
    if (p.rows >= 32 * sms) return forward_e<T, NARROW, 8, 4, kWarp, 128>(p, 32, 1, st);
    return forward_e<T, NARROW, 8, 1, kWarp, 128>(p, 32, 1, st);
  }
  constexpr size_t kOneCta = sizeof(T) == 2 ? 65536 : 32768;
  int c = cluster_for(p.rows, p.cols, 16384, sms);
  if (p.cols <= kOneCta && p.rows >= sms) c = 1;
  const size_t slice = div_up(p.cols, c);
  const bool few = p.rows * c <= 2 * sms && slice <= 4096;
  if (c > 1) {
    if (few) return forward_e<T, NARROW, 8, 1, kCluster, 512>(p, threads_for(slice, 8), c, st);
    return forward_e<T, NARROW, 32, 1, kCluster, 512>(p, threads_for(slice, 32), c, st);
  }
  if (few) return forward_e<T, NARROW, 8, 1, kCta, 512>(p, threads_for(slice, 8), 1, st);
  if (p.cols <= 512) return forward_e<T, NARROW, 16, 1, kWarp, 128>(p, 32, 1, st);
  if (p.cols <= 1024) return forward_e<T, NARROW, 32, 1, kWarp, 128>(p, 32, 1, st);
  if constexpr (sizeof(T) == 2) {
    if (p.cols <= 1792) return forward_e<T, NARROW, 64, 1, kWarp, 128>(p, 32, 1, st);
    if (p.cols > 2048 && p.cols <= 2 * 32 * 40) return forward_e<T, NARROW, 40, 1, kCta, 512>(p, 64, 1, st);
    if (p.cols > 4096 && p.cols <= 4 * 32 * 40) return forward_e<T, NARROW, 40, 1, kCta, 512>(p, 128, 1, st);
    if (p.cols > 4096 && p.cols <= 16384 && p.rows >= 4 * sms) return forward_e<T, NARROW, 64, 1, kCta, 512>(p, threads_for(slice, 64), 1, st);
  }
  if (p.cols <= 16384) return forward_e<T, NARROW, 32, 1, kCta, 512>(p, threads_for(slice, 32), 1, st);
  return forward_e<T, NARROW, sizeof(T) == 2 ? 64 : 32, 1, kCta, 1024>(p, threads_for(slice, sizeof(T) == 2 ? 64 : 32), 1, st);
}

// The shape of a backward launch, from the sizes alone (the workspace depends
// on it).  A thread has 16 columns (8 in rows of 256 and fewer): with their
// sums and gamma they take 48 registers, which leaves room for what is in
// work.  One CTA of up to 512 threads is on an SM, with as many rows side by
// side as it has room for, and leaves one partial sum per column; rows beyond
// 8192 columns are split over a cluster, and beyond 65536 a thread has 32.
// Rows up to 128 columns take half a warp each (200000 x 64 bf16: 26 us, 43 with whole
// warps; 100000 x 128: 22, 28).
//   Measured at 24576 x 5120 bf16 (755 MB), the kernel without the parts' sum:
//   118 us, 6.4 TB/s; 2 rows a turn 128, 1 row 136; 8 columns per thread, 640
//   threads and 4 rows 133; 24 columns, 224 threads and 1 row 175.  In
//   NARROW's layout 9973 x 1031 takes 29 us with 2 rows, 32 with 4 (the code
//   of a turn outgrows the instruction cache) and 35 with 1.
int resident_clusters(int csize);
BackwardShape backward_shape(size_t rows, size_t cols) {
  const size_t sms = sm_count();
  BackwardShape s;
  s.csize = cols <= 512 ? 1 : cluster_for(rows, cols, 512 * 16, sms);
  const size_t slice = div_up(cols, s.csize);
  s.e = slice <= 256 ? 8 : slice <= 8192 ? 16 : 32;
  s.threads = cols <= 128 ? 16 : threads_for(slice, s.e);
  s.groups = s.csize > 1 ? 1 : 512 / s.threads;
  if (s.threads > 32 && s.groups > 15) s.groups = 15;   // named barriers
  while (s.groups > 1 && div_up(rows, s.groups) < sms) s.groups /= 2;   // few rows: an SM each
  if (s.threads == 16 && s.groups == 1) s.threads = 32;   // a whole warp
  const size_t most = s.csize == 1 ? sms : (size_t)resident_clusters(s.csize);
  s.many = s.e <= 16 && rows >= 8 * s.groups * most;   // two turns for everyone at least
  const size_t want = div_up(rows, (size_t)s.groups);
  s.nparts = (unsigned)(want < most ? want : most);
  if (s.nparts < 1) s.nparts = 1;
  return s;
}

// Clusters of backward CTAs the GPU holds at once: fewer than its SMs would
// suggest, as a cluster lies within one GPC (of 152 SMs' worth of 5-CTA clusters, a second
// wave of a few doubles the time).
int resident_clusters(int csize) {
  static PerDevice known[kMaxCluster8 + 1];
  return known[csize].get([csize](int) {
    const auto kernel = ln_backward_kernel<bf16, false, 16, 1, kCluster>;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(csize);
    cfg.blockDim = dim3(512);
    cfg.dynamicSmemBytes = 200 * 1024;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = csize;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (allow_dynamic_smem(kernel) != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
      (void)cudaGetLastError();
      n = sm_count() / csize;
    }
    return n;
  });
}

template <typename T, bool NARROW, int E, int R, int MODE>
cudaError_t backward_e(NormRowsParams& p, const BackwardShape& s, cudaStream_t st) {
  p.threads = s.threads;
  p.nparts = s.nparts;
  constexpr int NV = E / kUnit<T>;
  const size_t stage = (size_t)s.groups * R * 2 * row_bytes<T, NARROW, NV>(s.threads);
  const size_t rest = (E > 16 ? (size_t)s.groups * E * s.threads * 4 : 0);
  const size_t acc = s.groups > 1 ? (size_t)2 * E * s.threads * 4 : 0;
  p.stages = stages_for(kSmemSm - 4096 - rest, stage, div_up(p.rows, (u64)s.nparts * s.groups * R));
  size_t smem = stage * p.stages + rest;
  if (smem < acc) smem = acc;
  return launch_dependent(ln_backward_kernel<T, NARROW, E, R, MODE>, dim3(s.nparts * s.csize), s.groups * s.threads, smem, s.csize, st, p);
}

// Rows a turn: 4, 2 or 1, as two stages of them fit in shared memory, or one
// in a cluster, whose barrier costs more than the loads it then waits for.
template <typename T, bool NARROW, int E, int MODE>
cudaError_t backward_r(NormRowsParams& p, const BackwardShape& s, cudaStream_t st) {
  const size_t row = (size_t)s.groups * 2 * row_bytes<T, NARROW, E / kUnit<T>>(s.threads);
  const size_t fit = (kSmemSm - 4096) / ((MODE == kCluster ? 1 : 2) * row);
  if constexpr (!NARROW && sizeof(T) == 2) {
    if (s.many && fit >= 4) return backward_e<T, NARROW, E, 4, MODE>(p, s, st);
  }
  if (s.many && fit >= 2) return backward_e<T, NARROW, E, 2, MODE>(p, s, st);
  return backward_e<T, NARROW, E, 1, MODE>(p, s, st);
}

template <typename T, bool NARROW>
cudaError_t backward(NormRowsParams& p, const BackwardShape& s, cudaStream_t st) {
  if (s.csize > 1) return s.e == 32 ? backward_e<T, NARROW, 32, 1, kCluster>(p, s, st) : backward_r<T, NARROW, 16, kCluster>(p, s, st);
  if (s.threads > 32) return backward_r<T, NARROW, 16, kCta>(p, s, st);
  if (s.threads == 16) {
    if constexpr (!NARROW) {
      return backward_r<T, NARROW, 8, kHalf>(p, s, st);
    } else {
      BackwardShape warps = s;
      warps.threads = 32;
      if (warps.groups > 16) warps.groups = 16;
      return backward_r<T, NARROW, 8, kWarp>(p, warps, st);
    }
  }
  return s.e == 8 ? backward_r<T, NARROW, 8, kWarp>(p, s, st) : backward_r<T, NARROW, 16, kWarp>(p, s, st);
}

bool wide_rows(const void* base, u64 stride, size_t cols, size_t esize) {
  return (reinterpret_cast<uintptr_t>(base) & 15u) == 0 && ((stride | cols) * esize & 15u) == 0;
}
bool wide_w(const void* w) { return (reinterpret_cast<uintptr_t>(w) & 15u) == 0; }

}  // namespace

cudaError_t launch_ln_forward(NormRowsParams& p, int dtype, cudaStream_t st) {
  const size_t es = dtype == XP_F32 ? 4 : 2;
  const bool wide = wide_rows(p.x, p.x_stride, p.cols, es) && wide_rows(p.out, p.out_stride, p.cols, es) && wide_w(p.gamma) && wide_w(p.beta);
  if (dtype == XP_F32) return wide ? forward<float, false>(p, st) : forward<float, true>(p, st);
  return wide ? forward<bf16, false>(p, st) : forward<bf16, true>(p, st);
}

BackwardShape ln_backward_shape(size_t rows, size_t cols) { return backward_shape(rows, cols); }

cudaError_t launch_ln_backward(NormRowsParams& p, const BackwardShape& s, int dtype, cudaStream_t st) {
  const size_t es = dtype == XP_F32 ? 4 : 2;
  const bool wide = wide_rows(p.x, p.x_stride, p.cols, es) && wide_rows(p.dy, p.dy_stride, p.cols, es) && wide_rows(p.out, p.out_stride, p.cols, es) && wide_w(p.gamma);
  cudaError_t e;
  if (dtype == XP_F32)
    e = wide ? backward<float, false>(p, s, st) : backward<float, true>(p, s, st);
  else
    e = wide ? backward<bf16, false>(p, s, st) : backward<bf16, true>(p, s, st);
  if (e != cudaSuccess || !p.dgamma || s.nparts == 1) return e;
  const bool four = p.cols % 4 == 0;   // and the workspace is aligned to 16 bytes
  return launch_dependent(four ? ln_parts_kernel<4> : ln_parts_kernel<1>, dim3((unsigned)div_up(p.cols, four ? 128 : 32), 2), 32 * kPartWarps,
                          0, 1, st, (const float*)p.partial, s.nparts, p.cols, p.dgamma, p.dbeta, p.accumulate);
}

}  // namespace xp
