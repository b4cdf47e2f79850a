// Layer norm, forward and backward, with the reduction of the weight's
// gradient over the rows.  include/xp_train.h states the formulas.
//
// Both directions read and write every element once and compute a handful of
// operations on it: HBM bounds them.  A row belongs to a group of threads
// that keeps it on chip between its sums and its output: a warp (short rows),
// a part of a CTA or a whole one, or the CTAs of a thread-block cluster, each
// with a slice of the row (long rows, and rows too few to fill the GPU).  A
// grid of as many CTAs as the GPU holds walks over the rows; asynchronous
// copies bring the next rows into shared memory while one is worked on.
#include "xp_train_device.cuh"

namespace xp {
namespace {

typedef __nv_bfloat16 bf16;
typedef unsigned long long u64;

// who shares a row
enum { kWarp = 0, kCta = 1, kCluster = 2 };
constexpr int kMaxWarps = 32;
constexpr int kMaxCluster8 = 8;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float f) { *p = f; }
__device__ __forceinline__ void put(bf16* p, float f) { *p = __float2bfloat16_rn(f); }

// ---- units: the V elements a thread takes at once.  Rows that allow it move
// in units of 16 bytes; others (lengths, strides or addresses that are no
// multiple of 16 bytes) in units of 4 bytes, one fp32 or two bf16, read from
// shared memory at any offset.
template <typename T, int V>
constexpr bool kWide = V * sizeof(T) == 16;

template <typename T, int V>
__device__ __forceinline__ void unpack16(uint4 q, float (&f)[V]) {
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
}
template <typename T, int V>
__device__ __forceinline__ uint4 pack16(const float (&f)[V]) {
  if constexpr (sizeof(T) == 4) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  } else {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    return *reinterpret_cast<uint4*>(h);
  }
}
// The first n elements of a unit (wide units are whole or absent) to global
// memory; p4: a 4-byte unit's address allows one store.
template <typename T, int V>
__device__ __forceinline__ void store_unit(T* p, int n, bool p4, const float (&f)[V]) {
  if constexpr (kWide<T, V>) {
    if (n > 0) *reinterpret_cast<uint4*>(p) = pack16<T, V>(f);
  } else if constexpr (V == 2) {
    if (n >= 2 && p4) {
      *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(f[0], f[1]);
    } else {
      if (n > 0) put(p, f[0]);
      if (n > 1) put(p + 1, f[1]);
    }
  } else {
    if (n > 0) put(p, f[0]);
  }
}
// gamma or beta: its own type, `none` where there is none
template <int V>
__device__ __forceinline__ void load_w(const void* w, int is_bf16, unsigned c, int n, float none, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = none;
  if (!w || n <= 0) return;
  if (is_bf16) {
    const bf16* p = static_cast<const bf16*>(w) + c;
    if constexpr (V == 8) {
      if (n >= V) return unpack16<bf16, V>(__ldg(reinterpret_cast<const uint4*>(p)), f);
    } else if constexpr (V == 4) {
      if (n >= V) {
        const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
        f[0] = __uint_as_float(q.x << 16);
        f[1] = __uint_as_float(q.x & 0xffff0000u);
        f[2] = __uint_as_float(q.y << 16);
        f[3] = __uint_as_float(q.y & 0xffff0000u);
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) f[i] = __bfloat162float(p[i]);
  } else {
    const float* p = static_cast<const float*>(w) + c;
    if constexpr (V >= 4) {
      if (n >= V) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
          const float4 q = __ldg(reinterpret_cast<const float4*>(p) + i);
          f[4 * i] = q.x;
          f[4 * i + 1] = q.y;
          f[4 * i + 2] = q.z;
          f[4 * i + 3] = q.w;
        }
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) f[i] = __ldg(p + i);
  }
}

// ---- sums over the threads of a row
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
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
__device__ __forceinline__ void store_remote(const float2* p, unsigned rank, float2 v) {
  unsigned a = (unsigned)__cvta_generic_to_shared(p), r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(r), "f"(v.x), "f"(v.y) : "memory");
}

// Shared words of the sums.  Two buffers in turn: a thread that reads one
// meets the others at the next sum's barrier before it is written again.
struct SumWords {
  float2 warp[2][kMaxWarps];
  float2 cta[2][kMaxCluster8];
};

// Both components summed over the row's threads, the same value in each; the
// order of the additions is fixed.  In steps, so that several rows share a
// barrier: each warp's sum, the group meets, the warps' sums added up; in a
// cluster then the same among its CTAs, through their shared memory.
template <int MODE>
__device__ __forceinline__ float2 row_partial(float2 v, SumWords& w, int buf) {
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  if (MODE != kWarp && (threadIdx.x & 31) == 0) w.warp[buf][threadIdx.x >> 5] = v;
  return v;
}
template <int MODE>
__device__ __forceinline__ void row_meet(int group, int threads) {
  if constexpr (MODE == kCluster) __syncthreads();
  if constexpr (MODE == kCta) group_bar(group, threads);
}
template <int MODE>
__device__ __forceinline__ float2 row_total(float2 v, const SumWords& w, int buf, int group, int threads) {
  if constexpr (MODE != kWarp) {
    const int lane = threadIdx.x & 31, nw = threads >> 5;
    v = lane < nw ? w.warp[buf][group * nw + lane] : make_float2(0.f, 0.f);
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
  }
  return v;
}
__device__ __forceinline__ void row_send(float2 v, SumWords& w, int buf) {
  if (threadIdx.x < cluster_size()) store_remote(&w.cta[buf][cluster_rank()], threadIdx.x, v);
}
__device__ __forceinline__ float2 row_join(const SumWords& w, int buf, unsigned n) {
  float2 v = make_float2(0.f, 0.f);
  for (unsigned r = 0; r < n; ++r) {
    v.x += w.cta[buf][r].x;
    v.y += w.cta[buf][r].y;
  }
  return v;
}
template <int MODE>
__device__ __forceinline__ float2 row_sum(float2 v, SumWords& w, int buf, int group, int threads) {
  v = row_partial<MODE>(v, w, buf);
  row_meet<MODE>(group, threads);
  v = row_total<MODE>(v, w, buf, group, threads);
  if constexpr (MODE == kCluster) {
    row_send(v, w, buf);
    cluster_arrive();
    cluster_wait();
    v = row_join(w, buf, cluster_size());
  }
  return v;
}

// ---- rows on their way from global to shared memory
__device__ __forceinline__ void copy_async16(unsigned smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}
// the first `bytes` of them, zeros after
__device__ __forceinline__ void copy_async16(unsigned smem, const void* gmem, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(bytes) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the newest n groups of this thread's copies have landed
__device__ __forceinline__ void wait_groups(int n) {
  switch (n) {
    case 0: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 1: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
    case 4: asm volatile("cp.async.wait_group 4;" ::: "memory"); break;
    case 5: asm volatile("cp.async.wait_group 5;" ::: "memory"); break;
    case 6: asm volatile("cp.async.wait_group 6;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 7;" ::: "memory"); break;
  }
}
constexpr int kMaxStages = 8;

// Bytes of shared memory that one row (one CTA's slice of it) takes.
template <typename T, int V>
__host__ __device__ constexpr unsigned row_bytes(unsigned threads, unsigned e) {
  return kWide<T, V> ? e * threads * (unsigned)sizeof(T) : (e * threads * (unsigned)sizeof(T) + 48u) & ~15u;
}

// One matrix's rows, as the threads of a group see them.  Past a row's end
// they read zeros.
//
// Wide units: a thread copies the units it will use itself, unit k at slot
// k * threads + thread, so nothing but its own copies has to have landed; it
// clears the slots of units that the row does not have once.
//
// 4-byte units: the group copies the 16-byte pieces that cover the row, at
// the row's own offset within them, and zeros behind them up to what a row at
// the largest offset would touch; the group meets before it reads.  A first
// piece that begins before the matrix does is copied element by element.
template <typename T, int V>
struct Rows {
  const T* base;      // row 0, first column of this CTA's slice
  u64 stride;
  const T* lo;        // the matrix's first element
  int cols;           // of the slice

  __device__ __forceinline__ const T* row(u64 r) const { return base + r * stride; }

  __device__ __forceinline__ void fetch_unit(const T* a, unsigned smem, int u) const {
    if (u * V < cols) copy_async16(smem + u * 16, a + u * V);
  }
  __device__ __forceinline__ void fetch_pieces(u64 r, char* smem, int tid, int threads) const {
    const char* a = reinterpret_cast<const char*>(row(r));
    const int len = cols * (int)sizeof(T), off = (int)(reinterpret_cast<uintptr_t>(a) & 15u);
    const char* first = a - off;
    const char* nothing = reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(lo) & ~(uintptr_t)15);   // of which 0 bytes are read
    const int pieces = (len + 29) >> 4;
    const unsigned to = (unsigned)__cvta_generic_to_shared(smem);
    for (int j = tid; j < pieces; j += threads) {
      const int here = min(max(off + len - 16 * j, 0), 16);   // bytes of this piece up to the row's end
      if (j == 0 && first < reinterpret_cast<const char*>(lo)) {
        for (int b = 0; b < 16; b += sizeof(T))
          *reinterpret_cast<T*>(smem + b) = b >= off && b < here ? *reinterpret_cast<const T*>(first + b) : T(0.f);
      } else {
        copy_async16(to + 16 * j, here ? first + 16 * j : nothing, here);
      }
    }
  }
  // Unit u of row r.
  __device__ __forceinline__ void read(u64 r, const char* smem, int u, float (&f)[V]) const {
    if constexpr (kWide<T, V>) {
      unpack16<T, V>(*reinterpret_cast<const uint4*>(smem + 16 * u), f);
    } else {
      const unsigned off = (unsigned)(reinterpret_cast<uintptr_t>(row(r)) & 15u);
      const unsigned* w = reinterpret_cast<const unsigned*>(smem + (off & ~3u)) + u;
      if constexpr (V == 1) {
        f[0] = __uint_as_float(w[0]);
      } else {
        unsigned q = w[0];
        if (off & 2) q = __byte_perm(q, w[1], 0x5432);
        f[0] = __uint_as_float(q << 16);
        f[1] = __uint_as_float(q & 0xffff0000u);
      }
    }
  }
};

// Clears what no copy will ever write: a thread's slots of units its rows do
// not have, or (4-byte units) all of the group's `bytes`.
template <typename T, int V, int NV>
__device__ __forceinline__ void clear_slots(char* slot, unsigned row_len, int nrows, int cols, int tid, int threads) {
  const uint4 zero = make_uint4(0, 0, 0, 0);
  if constexpr (kWide<T, V>) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int u = k * threads + tid;
      if (u * V >= cols)
        for (int r = 0; r < nrows; ++r) *reinterpret_cast<uint4*>(slot + r * row_len + 16 * u) = zero;
    }
  } else {
    for (unsigned b = 16 * tid; b < nrows * row_len; b += 16 * threads) *reinterpret_cast<uint4*>(slot + b) = zero;
  }
}

template <int MODE>
__device__ __forceinline__ void group_sync(int group, int threads) {
  if constexpr (MODE == kWarp)
    __syncwarp();
  else
    group_bar(group, threads);
}

// ---------------------------------------------------------------- forward

// The row stays in registers between its sums: E elements per thread, its
// unit k at column (k * threads + thread) * V.
template <typename T, int V, int E, int MODE, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) ln_forward_kernel(const __grid_constant__ NormRowsParams prm) {
  extern __shared__ uint4 s_dyn[];
  __shared__ SumWords words;
  constexpr int NV = E / V;
  constexpr bool WIDE = kWide<T, V>;
  const int threads = MODE == kWarp ? 32 : prm.threads;
  const int group = MODE == kCluster ? 0 : threadIdx.x / threads;
  const int tid = threadIdx.x - group * threads;
  const int groups = MODE == kCluster ? 1 : blockDim.x / threads;
  const unsigned csize = MODE == kCluster ? cluster_size() : 1;
  const unsigned c0 = MODE == kCluster ? cluster_rank() * E * threads : 0;
  const int cols = c0 < prm.cols ? (int)min((unsigned)E * threads, prm.cols - c0) : 0;   // a cluster's last CTA may have none
  const int stages = prm.stages;
  const unsigned len = row_bytes<T, V>(threads, E);
  char* slot = reinterpret_cast<char*>(s_dyn) + (size_t)group * stages * len;   // [group][stage]
  const unsigned slot_s = (unsigned)__cvta_generic_to_shared(slot);
  const Rows<T, V> x = {static_cast<const T*>(prm.x) + c0, prm.x_stride, static_cast<const T*>(prm.x), cols};
  const u64 step = (u64)(gridDim.x / csize) * groups;
  const u64 first = (u64)(blockIdx.x / csize) * groups + group;
  if (MODE == kCluster) cluster_arrive();   // its end: every CTA of the cluster runs
  clear_slots<T, V, NV>(slot, len, stages, cols, tid, threads);
  if constexpr (!WIDE) group_sync<MODE>(group, threads);
  wait_for_predecessors();
  let_successor_start();

  auto fetch = [&](u64 row, int stage) {
    if (row < prm.rows) {
      if constexpr (WIDE) {
#pragma unroll
        for (int k = 0; k < NV; ++k) x.fetch_unit(x.row(row), slot_s + stage * len, k * threads + tid);
      } else {
        x.fetch_pieces(row, slot + stage * len, tid, threads);
      }
    }
    commit();
  };
  for (int s = 0; s < stages; ++s) fetch(first + s * step, s);
  float g[E], b[E];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * threads + tid) * V;
    float w[V];
    load_w<V>(prm.gamma, prm.gamma_bf16, c0 + c, cols - c, 1.f, w);
#pragma unroll
    for (int i = 0; i < V; ++i) g[k * V + i] = w[i];
    load_w<V>(prm.beta, prm.gamma_bf16, c0 + c, cols - c, 0.f, w);
#pragma unroll
    for (int i = 0; i < V; ++i) b[k * V + i] = w[i];
  }
  if (MODE == kCluster) cluster_wait();
  const float inv = 1.0f / (float)prm.cols;
  int stage = 0;
  for (u64 row = first; row < prm.rows; row += step) {
    wait_groups(stages - 1);
    if constexpr (!WIDE) group_sync<MODE>(group, threads);   // the others' copies have landed too
    float f[NV][V];
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      x.read(row, slot + stage * len, k * threads + tid, f[k]);
#pragma unroll
      for (int i = 0; i < V; ++i) sum += f[k][i];
    }
    const float mean = row_sum<MODE>(make_float2(sum, 0.f), words, 0, group, threads).x * inv;
    // the row has been read: by this thread (wide units), or by the whole group (that met in the sum)
    if (!WIDE && MODE == kWarp) __syncwarp();
    fetch(row + (u64)stages * step, stage);
    if (++stage == stages) stage = 0;
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int n = cols - (k * threads + tid) * V;   // wide units are whole or absent
      const float m = n > 0 ? mean : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        f[k][i] -= WIDE || i < n ? m : 0.f;
        sq = fmaf(f[k][i], f[k][i], sq);
      }
    }
    const float var = row_sum<MODE>(make_float2(sq, 0.f), words, 1, group, threads).x * inv;
    const float rstd = 1.0f / sqrtf(var + prm.eps);
    if (tid == 0 && c0 == 0) {
      if (prm.mean) prm.mean[row] = mean;
      if (prm.rstd) prm.rstd[row] = rstd;
    }
    T* y = static_cast<T*>(prm.out) + row * prm.out_stride + c0;
    const bool p4 = (reinterpret_cast<uintptr_t>(y) & 3u) == 0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * threads + tid) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) f[k][i] = fmaf(f[k][i] * rstd, g[k * V + i], b[k * V + i]);
      store_unit<T, V>(y + c, cols - c, p4, f[k]);
    }
  }
}

// ---------------------------------------------------------------- backward

// Each group walks over its rows, R at a time, and keeps its columns' sums of
// dgamma and dbeta in registers.  A row is read twice from shared memory,
// for its sums and for dx: with d = x - mean and a = dy * gamma,
//   dx = rstd a - rstd sum(a) / cols - d rstd^3 sum(a d) / cols,
// dgamma += (dy rstd) d, dbeta += dy.
template <typename T, int V, int E, int R, int MODE, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) ln_backward_kernel(const __grid_constant__ NormRowsParams prm) {
  extern __shared__ uint4 s_dyn[];
  __shared__ SumWords words[R];
  constexpr int NV = E / V;
  constexpr bool WIDE = kWide<T, V>;
  constexpr bool kKeepGamma = E <= 16;                   // else in shared memory, a unit per thread as the rows'
  const int threads = MODE == kWarp ? 32 : prm.threads;
  const int group = MODE == kCluster ? 0 : threadIdx.x / threads;
  const int tid = threadIdx.x - group * threads;
  const int groups = MODE == kCluster ? 1 : blockDim.x / threads;
  const unsigned csize = MODE == kCluster ? cluster_size() : 1;
  const unsigned part = blockIdx.x / csize;
  const unsigned width = E * threads;                    // columns of a CTA
  const unsigned c0 = MODE == kCluster ? cluster_rank() * width : 0;
  const int cols = c0 < prm.cols ? (int)min(width, prm.cols - c0) : 0;   // a cluster's last CTA may have none
  const float inv = 1.0f / (float)prm.cols;
  const int stages = prm.stages;
  const unsigned len = row_bytes<T, V>(threads, E);
  char* slot = reinterpret_cast<char*>(s_dyn) + (size_t)group * stages * R * 2 * len;   // [group][stage][r][x, dy]
  const unsigned slot_s = (unsigned)__cvta_generic_to_shared(slot);
  const Rows<T, V> xr = {static_cast<const T*>(prm.x) + c0, prm.x_stride, static_cast<const T*>(prm.x), cols};
  const Rows<T, V> dr = {static_cast<const T*>(prm.dy) + c0, prm.dy_stride, static_cast<const T*>(prm.dy), cols};
  const u64 step = (u64)prm.nparts * groups * R;
  const u64 first = ((u64)part * groups + group) * R;
  clear_slots<T, V, NV>(slot, len, stages * R * 2, cols, tid, threads);
  if constexpr (!WIDE) group_sync<MODE>(group, threads);
  wait_for_predecessors();
  let_successor_start();

  auto fetch_piecewise = [&](u64 row, int stage) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row + r < prm.rows) {
        xr.fetch_pieces(row + r, slot + ((stage * R + r) * 2) * len, tid, threads);
        dr.fetch_pieces(row + r, slot + ((stage * R + r) * 2 + 1) * len, tid, threads);
      }
    }
    commit();
  };
  auto fetch_units = [&](const T* x, const T* dy, int stage, int r, int k) {
    xr.fetch_unit(x, slot_s + ((stage * R + r) * 2) * len, k * threads + tid);
    dr.fetch_unit(dy, slot_s + ((stage * R + r) * 2 + 1) * len, k * threads + tid);
  };
  for (int s = 0; s < stages; ++s) {
    if constexpr (WIDE) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const u64 row = first + s * step + r;
        if (row < prm.rows) {
#pragma unroll
          for (int k = 0; k < NV; ++k) fetch_units(xr.row(row), dr.row(row), s, r, k);
        }
      }
      commit();
    } else {
      fetch_piecewise(first + s * step, s);
    }
  }

  float dg[E], db[E];
#pragma unroll
  for (int i = 0; i < E; ++i) dg[i] = db[i] = 0.f;
  float gam[kKeepGamma ? E : 1];
  float* s_gam = reinterpret_cast<float*>(reinterpret_cast<char*>(s_dyn) + (size_t)groups * stages * R * 2 * len) + group * width;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * threads + tid) * V;
    float w[V];
    load_w<V>(prm.gamma, prm.gamma_bf16, c0 + c, cols - c, 1.f, w);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (kKeepGamma)
        gam[k * V + i] = w[i];
      else
        s_gam[c + i] = w[i];   // read back by this thread alone
    }
  }
  auto gammas = [&](int k, float (&w)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if constexpr (kKeepGamma) w[i] = gam[k * V + i];
    }
    if constexpr (!kKeepGamma) {
      const float* p = s_gam + (k * threads + tid) * V;
      if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
          const float4 q = *reinterpret_cast<const float4*>(p + i);
          w[i] = q.x, w[i + 1] = q.y, w[i + 2] = q.z, w[i + 3] = q.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) w[i] = p[i];
      }
    }
  };
  float mean_next[R], rstd_next[R];
  auto statistics = [&](u64 row) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      mean_next[r] = row + r < prm.rows ? __ldg(prm.mean + row + r) : 0.f;
      rstd_next[r] = row + r < prm.rows ? __ldg(prm.rstd + row + r) : 0.f;
    }
  };
  statistics(first);
  if (MODE == kCluster) {   // every CTA of the cluster runs before its shared memory is written
    cluster_arrive();
    cluster_wait();
  }
  int stage = 0, last = 0, buf = 0;
  for (u64 row = first; row < prm.rows; row += step) {
    float mean[R], rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) mean[r] = mean_next[r], rstd[r] = rstd_next[r];
    statistics(row + step);
    // the group of copies for these rows: the newest but stages - 1, and one newer where they were asked for a turn later
    wait_groups(WIDE ? stages - 1 : stages > 2 ? stages - 2 : 0);
    if constexpr (!WIDE) group_sync<MODE>(group, threads);   // the others' copies have landed too
    const char* here = slot + stage * R * 2 * len;
    float2 s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] = make_float2(0.f, 0.f);
      if (row + r < prm.rows) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          float fx[V], fd[V], w[V];
          xr.read(row + r, here + r * 2 * len, k * threads + tid, fx);
          dr.read(row + r, here + (r * 2 + 1) * len, k * threads + tid, fd);
          gammas(k, w);
#pragma unroll
          for (int i = 0; i < V; ++i) {   // dy is 0 past the row's end
            const float d = fx[i] - mean[r], a = fd[i] * w[i];
            s[r].x += a;
            s[r].y = fmaf(a, d, s[r].y);
            dg[k * V + i] = fmaf(fd[i] * rstd[r], d, dg[k * V + i]);
            db[k * V + i] += fd[i];
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = row_partial<MODE>(s[r], words[r], buf);
    row_meet<MODE>(group, threads);
#pragma unroll
    for (int r = 0; r < R; ++r) s[r] = row_total<MODE>(s[r], words[r], buf, group, threads);
    if constexpr (MODE == kCluster) {
#pragma unroll
      for (int r = 0; r < R; ++r) row_send(s[r], words[r], buf);
      cluster_arrive();
      cluster_wait();
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] = row_join(words[r], buf, csize);
    }
    buf ^= 1;
    // 4-byte units: the group has met since it read the previous rows for dx, so their slots are free
    if constexpr (!WIDE) {
      if (stages > 1 && row != first) fetch_piecewise(row + (u64)(stages - 1) * step, last);
      else commit();
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (row + r < prm.rows) {
        T* dx = static_cast<T*>(prm.out) + (row + r) * prm.out_stride + c0;
        const bool p4 = (reinterpret_cast<uintptr_t>(dx) & 3u) == 0;
        const u64 next = row + (u64)stages * step + r;
        const T *x_next = xr.row(next), *dy_next = dr.row(next);
        const float k1 = -rstd[r] * (s[r].x * inv);
        const float k2 = -rstd[r] * rstd[r] * rstd[r] * (s[r].y * inv);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int c = (k * threads + tid) * V;
          float fx[V], fd[V], w[V];
          xr.read(row + r, here + r * 2 * len, k * threads + tid, fx);
          dr.read(row + r, here + (r * 2 + 1) * len, k * threads + tid, fd);
          if constexpr (WIDE) {   // this unit's slot is free
            if (next < prm.rows) fetch_units(x_next, dy_next, stage, r, k);
          }
          gammas(k, w);
#pragma unroll
          for (int i = 0; i < V; ++i) fd[i] = fmaf(fx[i] - mean[r], k2, fmaf(fd[i] * w[i], rstd[r], k1));
          store_unit<T, V>(dx + c, cols - c, p4, fd);
        }
      }
    }
    if constexpr (WIDE) {
      commit();
    } else if (stages == 1) {
      group_sync<MODE>(group, threads);
      fetch_piecewise(row + step, 0);
    }
    last = stage;
    if (++stage == stages) stage = 0;
  }
  wait_groups(0);
  if (!prm.dgamma) return;

  // the groups' sums, added in their order, then one part of the CTA or cluster
  float* out_g = (prm.nparts > 1 ? prm.partial + (size_t)part * 2 * prm.cols : prm.dgamma) + c0;
  float* out_b = (prm.nparts > 1 ? prm.partial + ((size_t)part * 2 + 1) * prm.cols : prm.dbeta) + c0;
  const bool add = prm.nparts == 1 && prm.accumulate;
  if (groups > 1) {
    float* acc = reinterpret_cast<float*>(s_dyn);   // [2][width]
    for (int g = 0; g < groups; ++g) {
      __syncthreads();
      if (g != group) continue;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = (k * threads + tid) * V + i;
          acc[c] = g ? acc[c] + dg[k * V + i] : dg[k * V + i];
          acc[width + c] = g ? acc[width + c] + db[k * V + i] : db[k * V + i];
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
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (k * threads + tid) * V + i;
        if (c < cols) {
          out_g[c] = add ? out_g[c] + dg[k * V + i] : dg[k * V + i];
          out_b[c] = add ? out_b[c] + db[k * V + i] : db[k * V + i];
        }
      }
    }
  }
}

// The parts' sums, column by column: 32 columns per CTA, 16 warps that each
// add every 16th part in fp64, then the warps' sums in order.
constexpr int kPartWarps = 16;
__global__ void __launch_bounds__(32 * kPartWarps) ln_parts_kernel(const float* partial, unsigned nparts, unsigned cols,
                                                                  float* dgamma, float* dbeta, int accumulate) {
  __shared__ double s[kPartWarps][32];
  wait_for_predecessors();
  let_successor_start();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned c = blockIdx.x * 32 + lane;
  const float* p = partial + (size_t)blockIdx.y * cols + c;
  double sum = 0.0;
  if (c < cols) {
    unsigned k = warp;
    for (; k + 3 * kPartWarps < nparts; k += 4 * kPartWarps) {
      const float a0 = p[(size_t)k * 2 * cols], a1 = p[(size_t)(k + kPartWarps) * 2 * cols];
      const float a2 = p[(size_t)(k + 2 * kPartWarps) * 2 * cols], a3 = p[(size_t)(k + 3 * kPartWarps) * 2 * cols];
      sum += ((double)a0 + a1) + ((double)a2 + a3);
    }
    for (; k < nparts; k += kPartWarps) sum += p[(size_t)k * 2 * cols];
  }
  s[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && c < cols) {
    for (int w = 1; w < kPartWarps; ++w) sum += s[w][lane];
    float* out = (blockIdx.y ? dbeta : dgamma) + c;
    *out = accumulate ? *out + (float)sum : (float)sum;
  }
}

// ---------------------------------------------------------------- launches

int sm_count() {
  static const int n = [] {
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v < 1) {
      (void)cudaGetLastError();
      v = 152;
    }
    return v;
  }();
  return n;
}

size_t div_up(size_t a, size_t b) { return (a + b - 1) / b; }
int threads_for(size_t elems, int e) { return elems ? 32 * (int)div_up(elems, (size_t)32 * e) : 32; }

// A row's CTAs: enough that a slice fits, and more where the rows are too few
// for the GPU's SMs, as long as a slice keeps 2048 columns.
int cluster_for(size_t rows, size_t cols, size_t most) {
  int c = 1;
  while (c < kMaxCluster8 && (div_up(cols, c) > most || (rows * c < (size_t)sm_count() && cols / (2 * c) >= 2048))) c *= 2;
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

constexpr size_t kSmemSm = 224 * 1024;   // of an SM, less what CTAs take statically

template <typename T, int V, int E, int MODE, int MAXT, int MINB>
cudaError_t forward_e(NormRowsParams& p, int threads, int csize, cudaStream_t st) {
  const int groups = MODE == kCluster ? 1 : MAXT / threads > 15 && MODE == kCta ? 15 : MAXT / threads;
  const size_t want = div_up(p.rows, groups), most = (size_t)MINB * sm_count() / csize;
  const unsigned n = (unsigned)(want < most ? want : most);
  p.threads = threads;
  const size_t row = (size_t)groups * row_bytes<T, V>(threads, E);
  p.stages = stages_for(kSmemSm / MINB - 2048, row, div_up(want, n));
  return launch_dependent(ln_forward_kernel<T, V, E, MODE, MAXT, MINB>, n * csize, groups * threads, row * p.stages, csize, st, p);
}

template <typename T, int V>
cudaError_t forward(NormRowsParams& p, cudaStream_t st) {
  if (p.cols <= 512) return forward_e<T, V, 16, kWarp, 256, 3>(p, 32, 1, st);
  const int c = cluster_for(p.rows, p.cols, 1024 * 16);
  const int threads = threads_for(div_up(p.cols, c), 16);
  if (c > 1) return threads <= 256 ? forward_e<T, V, 16, kCluster, 256, 3>(p, threads, c, st) : forward_e<T, V, 16, kCluster, 1024, 1>(p, threads, c, st);
  return threads <= 256 ? forward_e<T, V, 16, kCta, 256, 3>(p, threads, 1, st) : forward_e<T, V, 16, kCta, 1024, 1>(p, threads, 1, st);
}

// The shape of a backward launch, from the sizes alone (the workspace depends
// on it).  Up to 8192 columns a CTA has 256 threads, so that two to four are
// on an SM and one's barrier is another's work.
struct BackwardShape {
  int e, r, threads, groups, csize, ctas;   // ctas: per SM
  unsigned nparts;
};
BackwardShape backward_shape(size_t rows, size_t cols) {
  BackwardShape s;
  s.csize = cols <= 256 ? 1 : cluster_for(rows, cols, 512 * 32);
  const size_t slice = div_up(cols, s.csize);
  s.e = slice <= 2048 ? 8 : slice <= 4096 ? 16 : slice <= 6144 ? 24 : 32;
  s.threads = threads_for(slice, s.e);
  s.r = s.e <= 16 ? 2 : 1;
  s.ctas = slice > 8192 ? 1 : s.e == 8 ? 3 : 2;
  s.groups = s.csize > 1 || s.threads > 256 ? 1 : 256 / s.threads;
  const size_t want = div_up(rows, (size_t)s.groups * s.r), most = (size_t)s.ctas * sm_count() / s.csize;
  s.nparts = (unsigned)(want < most ? want : most);
  if (s.nparts < 1) s.nparts = 1;
  return s;
}

template <typename T, int V, int E, int R, int MODE, int MAXT, int MINB>
cudaError_t backward_e(NormRowsParams& p, const BackwardShape& s, cudaStream_t st) {
  p.threads = s.threads;
  p.nparts = s.nparts;
  const size_t stage = (size_t)s.groups * R * 2 * row_bytes<T, V>(s.threads, E);
  const size_t gam = E > 16 ? (size_t)s.groups * E * s.threads * 4 : 0;
  const size_t acc = s.groups > 1 ? (size_t)2 * E * s.threads * 4 : 0;
  p.stages = stages_for(kSmemSm / MINB - 2048 - gam, stage, div_up(p.rows, (u64)s.nparts * s.groups * R));
  size_t smem = stage * p.stages + gam;
  if (smem < acc) smem = acc;
  return launch_dependent(ln_backward_kernel<T, V, E, R, MODE, MAXT, MINB>, s.nparts * s.csize, s.groups * s.threads, smem, s.csize, st, p);
}

template <typename T, int V>
cudaError_t backward(NormRowsParams& p, const BackwardShape& s, cudaStream_t st) {
  if (s.csize > 1) {
    if (s.e == 8) return backward_e<T, V, 8, 2, kCluster, 256, 3>(p, s, st);
    if (s.e == 16) return backward_e<T, V, 16, 2, kCluster, 256, 2>(p, s, st);
    if (s.e == 24) return backward_e<T, V, 24, 1, kCluster, 256, 2>(p, s, st);
    return s.threads <= 256 ? backward_e<T, V, 32, 1, kCluster, 256, 2>(p, s, st) : backward_e<T, V, 32, 1, kCluster, 512, 1>(p, s, st);
  }
  if (s.threads == 32) return backward_e<T, V, 8, 2, kWarp, 256, 3>(p, s, st);
  if (s.e == 8) return backward_e<T, V, 8, 2, kCta, 256, 3>(p, s, st);
  if (s.e == 16) return backward_e<T, V, 16, 2, kCta, 256, 2>(p, s, st);
  if (s.e == 24) return backward_e<T, V, 24, 1, kCta, 256, 2>(p, s, st);
  return s.threads <= 256 ? backward_e<T, V, 32, 1, kCta, 256, 2>(p, s, st) : backward_e<T, V, 32, 1, kCta, 512, 1>(p, s, st);
}

bool wide_rows(const void* base, u64 stride, size_t cols, size_t esize) {
  return (reinterpret_cast<uintptr_t>(base) & 15u) == 0 && ((stride | cols) * esize & 15u) == 0;
}
bool wide_w(const void* w) { return (reinterpret_cast<uintptr_t>(w) & 15u) == 0; }

}  // namespace

cudaError_t launch_ln_forward(NormRowsParams& p, int dtype, cudaStream_t st) {
  const size_t es = dtype == XP_F32 ? 4 : 2;
  const bool wide = wide_rows(p.x, p.x_stride, p.cols, es) && wide_rows(p.out, p.out_stride, p.cols, es) && wide_w(p.gamma) && wide_w(p.beta);
  if (dtype == XP_F32) return wide ? forward<float, 4>(p, st) : forward<float, 1>(p, st);
  return wide ? forward<bf16, 8>(p, st) : forward<bf16, 2>(p, st);
}

cudaError_t ln_backward_parts(size_t rows, size_t cols, unsigned* nparts) {
  *nparts = rows && cols ? backward_shape(rows, cols).nparts : 0;
  return cudaSuccess;
}

cudaError_t launch_ln_backward(NormRowsParams& p, int dtype, cudaStream_t st) {
  const size_t es = dtype == XP_F32 ? 4 : 2;
  const BackwardShape s = backward_shape(p.rows, p.cols);
  const bool wide = wide_rows(p.x, p.x_stride, p.cols, es) && wide_rows(p.dy, p.dy_stride, p.cols, es) && wide_rows(p.out, p.out_stride, p.cols, es) && wide_w(p.gamma);
  cudaError_t e;
  if (dtype == XP_F32)
    e = wide ? backward<float, 4>(p, s, st) : backward<float, 1>(p, s, st);
  else
    e = wide ? backward<bf16, 8>(p, s, st) : backward<bf16, 2>(p, s, st);
  if (e != cudaSuccess || !p.dgamma || s.nparts == 1) return e;
  return launch_dependent(ln_parts_kernel, dim3((unsigned)div_up(p.cols, 32), 2), 32 * kPartWarps, 0, 1, st, (const float*)p.partial, s.nparts,
                          p.cols, p.dgamma, p.dbeta, p.accumulate);
}

}  // namespace xp
