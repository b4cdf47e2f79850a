// Layer norm, forward and backward, with the reduction of the weight's
// gradient over the rows.  include/xp_train.h states the formulas.
//
// Both directions read and write every element once and compute a handful of
// operations on it: HBM bounds them.  A row belongs to a group of threads
// that keeps it on chip between its sums and its output: a warp (short rows),
// a part of a CTA or a whole one, or the CTAs of a thread-block cluster, each
// with a slice of the row (long rows, and rows too few to fill the GPU).
#include <cuda_bf16.h>

#include "xp_train_internal.h"

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

// ---- V elements at once: V * sizeof(T) = 16 bytes, or V = 1
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
template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, int n, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = n > 0 ? to_f(*p) : 0.f;
  } else if (n >= V) {
    unpack16<T, V>(*reinterpret_cast<const uint4*>(p), f);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = i < n ? to_f(p[i]) : 0.f;
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, int n, const float (&f)[V]) {
  if constexpr (V == 1) {
    if (n > 0) put(p, f[0]);
  } else if (n >= V) {
    *reinterpret_cast<uint4*>(p) = pack16<T, V>(f);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) put(p + i, f[i]);
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
// order of the additions is fixed.
template <int MODE>
__device__ __forceinline__ float2 row_sum(float2 v, SumWords& w, int buf, int group, int threads) {
  v.x = warp_sum(v.x);
  v.y = warp_sum(v.y);
  if constexpr (MODE != kWarp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = threads >> 5, first = group * nw;
    if (lane == 0) w.warp[buf][warp] = v;
    if (MODE == kCluster)
      __syncthreads();
    else
      group_bar(group, threads);
    v = lane < nw ? w.warp[buf][first + lane] : make_float2(0.f, 0.f);
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if constexpr (MODE == kCluster) {
      const unsigned n = cluster_size();
      if (threadIdx.x < n) store_remote(&w.cta[buf][cluster_rank()], threadIdx.x, v);
      cluster_arrive();
      cluster_wait();
      v = make_float2(0.f, 0.f);
      for (unsigned r = 0; r < n; ++r) {
        v.x += w.cta[buf][r].x;
        v.y += w.cta[buf][r].y;
      }
    }
  }
  return v;
}

// ---------------------------------------------------------------- forward

// The row stays in registers: E elements per thread, its vector k at column
// (k * threads + thread) * V.
template <typename T, int V, int E, int MODE>
__global__ void __launch_bounds__(MODE == kWarp ? 128 : 1024) ln_forward_kernel(const __grid_constant__ NormRowsParams prm) {
  __shared__ SumWords words;
  constexpr int NV = E / V;
  const int threads = MODE == kWarp ? 32 : blockDim.x;
  const int tid = MODE == kWarp ? threadIdx.x & 31 : threadIdx.x;
  const u64 row = MODE == kWarp      ? (u64)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)
                  : MODE == kCluster ? blockIdx.x / cluster_size()
                                     : blockIdx.x;
  if (MODE == kWarp && row >= prm.rows) return;
  if (MODE == kCluster) cluster_arrive();   // its end: every CTA of the cluster runs
  const unsigned c0 = MODE == kCluster ? cluster_rank() * prm.slice : 0;
  const int cols = (int)(MODE == kCluster ? min(prm.slice, prm.cols - c0) : prm.cols);
  const T* x = static_cast<const T*>(prm.x) + row * prm.x_stride + c0;

  float f[NV][V];
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) load_v<T, V>(x + (k * threads + tid) * V, cols - (k * threads + tid) * V, f[k]);
#pragma unroll
  for (int k = 0; k < NV; ++k) {
#pragma unroll
    for (int i = 0; i < V; ++i) sum += f[k][i];
  }
  if (MODE == kCluster) cluster_wait();
  const float mean = row_sum<MODE>(make_float2(sum, 0.f), words, 0, 0, threads).x / (float)prm.cols;
  float sq = 0.f;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int n = cols - (k * threads + tid) * V;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float d = i < n ? f[k][i] - mean : 0.f;
      sq += d * d;
    }
  }
  const float var = row_sum<MODE>(make_float2(sq, 0.f), words, 1, 0, threads).x / (float)prm.cols;
  const float rstd = 1.0f / sqrtf(var + prm.eps);
  if (tid == 0 && c0 == 0) {
    if (prm.mean) prm.mean[row] = mean;
    if (prm.rstd) prm.rstd[row] = rstd;
  }
  T* y = static_cast<T*>(prm.out) + row * prm.out_stride + c0;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = (k * threads + tid) * V, n = cols - c;
    float g[V], b[V];
    load_w<V>(prm.gamma, prm.gamma_bf16, c0 + c, n, 1.f, g);
    load_w<V>(prm.beta, prm.gamma_bf16, c0 + c, n, 0.f, b);
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = (f[k][i] - mean) * rstd * g[i] + b[i];
    store_v<T, V>(y + c, n, g);
  }
}

// ---------------------------------------------------------------- backward

__device__ __forceinline__ void copy_async16(void* smem, const void* gmem) {
  const unsigned s = (unsigned)__cvta_generic_to_shared(smem);
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(s), "l"(gmem) : "memory");
}
__device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the newest n groups have landed
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

// Each group walks over rows and keeps its columns' sums of dgamma and dbeta
// in registers.  V > 1: every thread copies the vectors it will use itself,
// some rows ahead, into slots of its own in shared memory, so no barrier
// guards them.
template <typename T, int V, int E, int MODE>
__global__ void __launch_bounds__(512) ln_backward_kernel(const __grid_constant__ NormRowsParams prm) {
  extern __shared__ uint4 s_rows[];
  __shared__ SumWords words;
  constexpr int NV = E / V;
  const int threads = MODE == kWarp ? 32 : prm.slice;   // slice: threads per row here
  const int group = MODE == kCluster ? 0 : threadIdx.x / threads;
  const int tid = threadIdx.x - group * threads;
  const int groups = blockDim.x / threads;
  const unsigned csize = MODE == kCluster ? cluster_size() : 1;
  const unsigned part = blockIdx.x / csize;
  const unsigned width = E * threads;                    // columns of a CTA
  const unsigned c0 = MODE == kCluster ? cluster_rank() * width : 0;
  const int cols = c0 < prm.cols ? (int)min(width, prm.cols - c0) : 0;   // 0: a cluster's last CTA may have none
  const float inv = 1.0f / (float)prm.cols;
  const bool staged = V > 1;
  const int stages = prm.stages;

  // thread's slots: [stage][group][x, dy][k][thread]
  uint4* slots = s_rows + (size_t)group * 2 * NV * threads + tid;
  const size_t stage_len = (size_t)groups * 2 * NV * threads;
  const u64 step = (u64)prm.nparts * groups;
  const u64 first = (u64)part * groups + group;

  auto fetch = [&](u64 row, int stage) {
    if constexpr (V > 1) {
      if (row < prm.rows) {
        const T* x = static_cast<const T*>(prm.x) + row * prm.x_stride + c0;
        const T* dy = static_cast<const T*>(prm.dy) + row * prm.dy_stride + c0;
        uint4* s = slots + stage * stage_len;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
          const int c = (k * threads + tid) * V;
          if (c + V <= cols) {
            copy_async16(s + k * threads, x + c);
            copy_async16(s + (NV + k) * threads, dy + c);
          }
        }
      }
      commit();
    }
  };
  // vector k of x and of dy; a row's last vector, if short, comes from global memory
  auto vectors = [&](u64 row, int stage, int k, float (&fx)[V], float (&fd)[V]) {
    const int c = (k * threads + tid) * V;
    if (staged && c + V <= cols) {
      if constexpr (V > 1) {
        const uint4* s = slots + stage * stage_len;
        unpack16<T, V>(s[k * threads], fx);
        unpack16<T, V>(s[(NV + k) * threads], fd);
      }
    } else {
      load_v<T, V>(static_cast<const T*>(prm.x) + row * prm.x_stride + c0 + c, min(cols - c, V > 1 ? V - 1 : 1), fx);
      load_v<T, V>(static_cast<const T*>(prm.dy) + row * prm.dy_stride + c0 + c, min(cols - c, V > 1 ? V - 1 : 1), fd);
    }
  };

  float dg[E], db[E];
#pragma unroll
  for (int i = 0; i < E; ++i) dg[i] = db[i] = 0.f;
  constexpr bool kKeepGamma = E <= 16;
  float gam[kKeepGamma ? E : 1];
  if constexpr (kKeepGamma) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * threads + tid) * V;
      float w[V];
      load_w<V>(prm.gamma, prm.gamma_bf16, c0 + c, cols - c, 1.f, w);
#pragma unroll
      for (int i = 0; i < V; ++i) gam[k * V + i] = w[i];
    }
  }
  auto gammas = [&](int k, float (&w)[V]) {
    if constexpr (kKeepGamma) {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = gam[k * V + i];
    } else {
      const int c = (k * threads + tid) * V;
      load_w<V>(prm.gamma, prm.gamma_bf16, c0 + c, cols - c, 1.f, w);
    }
  };

  for (int s = 0; s < stages; ++s) fetch(first + s * step, s);
  float mean_next = 0.f, rstd_next = 0.f;
  if (first < prm.rows) {
    mean_next = prm.mean[first];
    rstd_next = prm.rstd[first];
  }
  if (MODE == kCluster) {   // every CTA of the cluster runs before its shared memory is written
    cluster_arrive();
    cluster_wait();
  }
  int stage = 0, buf = 0;
  for (u64 row = first; row < prm.rows; row += step) {
    const float mean = mean_next, rstd = rstd_next;
    if (row + step < prm.rows) {
      mean_next = prm.mean[row + step];
      rstd_next = prm.rstd[row + step];
    }
    if (staged) wait_groups(stages - 1);
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      float fx[V], fd[V], w[V];
      vectors(row, stage, k, fx, fd);
      gammas(k, w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xhat = (fx[i] - mean) * rstd, a = fd[i] * w[i];   // dy is 0 past the row's end
        s.x += a;
        s.y += a * xhat;
        dg[k * V + i] += fd[i] * xhat;
        db[k * V + i] += fd[i];
      }
    }
    s = row_sum<MODE>(s, words, buf, group, threads);
    buf ^= 1;
    const float c1 = s.x * inv, c2 = s.y * inv;
    T* dx = static_cast<T*>(prm.out) + row * prm.out_stride + c0;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = (k * threads + tid) * V;
      float fx[V], fd[V], w[V];
      vectors(row, stage, k, fx, fd);
      gammas(k, w);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float xhat = (fx[i] - mean) * rstd;
        fd[i] = (fd[i] * w[i] - c1 - xhat * c2) * rstd;
      }
      store_v<T, V>(dx + c, cols - c, fd);
    }
    fetch(row + (u64)stages * step, stage);
    if (++stage == stages) stage = 0;
  }
  if (staged) wait_groups(0);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!prm.dgamma) return;

  // the groups' sums, added in their order, then one part of the CTA or cluster
  float* out_g = prm.nparts > 1 ? prm.partial + (size_t)part * 2 * prm.cols : prm.dgamma;
  float* out_b = prm.nparts > 1 ? out_g + prm.cols : prm.dbeta;
  const bool add = prm.nparts == 1 && prm.accumulate;
  if (groups > 1) {
    float* acc = reinterpret_cast<float*>(s_rows);   // [2][width]
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
          out_g[c0 + c] = add ? out_g[c0 + c] + dg[k * V + i] : dg[k * V + i];
          out_b[c0 + c] = add ? out_b[c0 + c] + db[k * V + i] : db[k * V + i];
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
  asm volatile("griddepcontrol.wait;" ::: "memory");
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

unsigned div_up(size_t a, size_t b) { return (unsigned)((a + b - 1) / b); }
int warps_for(size_t elems, int e) { return (int)div_up(elems, (size_t)32 * e); }

template <typename K>
cudaError_t launch_k(K kernel, unsigned grid, int block, size_t smem, int csize, const NormRowsParams& p, cudaStream_t st) {
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  if (csize > 1) {
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = csize;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// A row's CTAs: enough that a slice fits, and more where the rows are too few
// for the GPU's SMs, as long as a slice keeps 2048 columns.
int cluster_for(size_t rows, size_t cols, size_t most) {
  int c = 1;
  while (c < kMaxCluster8 && ((cols + c - 1) / c > most || (rows * c < (size_t)sm_count() && cols / (2 * c) >= 2048))) c *= 2;
  return c;
}

template <typename T, int V>
cudaError_t forward(NormRowsParams& p, cudaStream_t st) {
  if (p.cols <= 32 * 8) {
    const int warps = 4;
    return launch_k(ln_forward_kernel<T, V, 8, kWarp>, div_up(p.rows, warps), 32 * warps, 0, 1, p, st);
  }
  const int c = cluster_for(p.rows, p.cols, 1024 * 16);
  if (c == 1) {
    if (p.cols <= 1024 * 8) return launch_k(ln_forward_kernel<T, V, 8, kCta>, (unsigned)p.rows, 32 * warps_for(p.cols, 8), 0, 1, p, st);
    return launch_k(ln_forward_kernel<T, V, 16, kCta>, (unsigned)p.rows, 32 * warps_for(p.cols, 16), 0, 1, p, st);
  }
  p.slice = div_up(div_up(p.cols, c), 8) * 8;
  const int used = (int)div_up(p.cols, p.slice);   // == c: a slice has 2048 columns at least
  if (p.slice <= 1024 * 8) return launch_k(ln_forward_kernel<T, V, 8, kCluster>, (unsigned)p.rows * used, 32 * warps_for(p.slice, 8), 0, used, p, st);
  return launch_k(ln_forward_kernel<T, V, 16, kCluster>, (unsigned)p.rows * used, 32 * warps_for(p.slice, 16), 0, used, p, st);
}

// The shape of a backward launch, from the sizes alone (the workspace depends on it).
struct BackwardShape {
  int e, threads, groups, csize;
  unsigned nparts;
};
BackwardShape backward_shape(size_t rows, size_t cols) {
  BackwardShape s;
  s.csize = cols <= 256 ? 1 : cluster_for(rows, cols, 512 * 32);
  const size_t slice = (cols + s.csize - 1) / s.csize;
  s.e = slice <= 4096 ? 8 : slice <= 8192 ? 16 : 32;
  s.threads = 32 * (warps_for(slice, s.e) < 1 ? 1 : warps_for(slice, s.e));
  s.groups = s.csize > 1 ? 1 : 512 / s.threads;
  if (s.groups > 15 && s.threads > 32) s.groups = 15;   // named barriers
  const size_t want = (rows + s.groups - 1) / s.groups, most = (size_t)(2 * sm_count()) / s.csize;
  s.nparts = (unsigned)(want < most ? want : most);
  if (s.nparts < 1) s.nparts = 1;
  return s;
}

template <typename T, int V, int E, int MODE>
cudaError_t backward_e(NormRowsParams& p, const BackwardShape& s, cudaStream_t st) {
  p.slice = s.threads;
  p.nparts = s.nparts;
  const size_t stage = V > 1 ? (size_t)s.groups * 2 * (E / V) * s.threads * 16 : 0;
  const size_t acc = s.groups > 1 ? (size_t)2 * E * s.threads * 4 : 0;
  p.stages = 1;
  if (stage) {
    const size_t budget = 100 * 1024;   // two CTAs per SM
    size_t n = budget / stage;
    p.stages = (int)(n < 1 ? 1 : n > kMaxStages ? kMaxStages : n);
    const u64 turns = (p.rows + (u64)s.nparts * s.groups - 1) / ((u64)s.nparts * s.groups);
    if ((u64)p.stages > turns) p.stages = (int)(turns ? turns : 1);
  }
  size_t smem = stage * p.stages;
  if (smem < acc) smem = acc;
  return launch_k(ln_backward_kernel<T, V, E, MODE>, s.nparts * s.csize, s.groups * s.threads, smem, s.csize, p, st);
}

template <typename T, int V>
cudaError_t backward(NormRowsParams& p, const BackwardShape& s, cudaStream_t st) {
  if (s.csize > 1) {
    if (s.e == 8) return backward_e<T, V, 8, kCluster>(p, s, st);
    if (s.e == 16) return backward_e<T, V, 16, kCluster>(p, s, st);
    return backward_e<T, V, 32, kCluster>(p, s, st);
  }
  if (s.threads == 32) return backward_e<T, V, 8, kWarp>(p, s, st);
  if (s.e == 8) return backward_e<T, V, 8, kCta>(p, s, st);
  if (s.e == 16) return backward_e<T, V, 16, kCta>(p, s, st);
  return backward_e<T, V, 32, kCta>(p, s, st);
}

bool vec_rows(const void* base, u64 stride, size_t esize) {
  return (reinterpret_cast<uintptr_t>(base) & 15u) == 0 && (stride * esize & 15u) == 0;
}
bool vec_w(const void* w) { return (reinterpret_cast<uintptr_t>(w) & 15u) == 0; }

}  // namespace

cudaError_t launch_ln_forward(NormRowsParams& p, int dtype, cudaStream_t st) {
  const size_t es = dtype == XP_F32 ? 4 : 2;
  const bool vec = vec_rows(p.x, p.x_stride, es) && vec_rows(p.out, p.out_stride, es) && vec_w(p.gamma) && vec_w(p.beta);
  if (dtype == XP_F32) return vec ? forward<float, 4>(p, st) : forward<float, 1>(p, st);
  return vec ? forward<bf16, 8>(p, st) : forward<bf16, 1>(p, st);
}

cudaError_t ln_backward_parts(size_t rows, size_t cols, unsigned* nparts) {
  *nparts = rows && cols ? backward_shape(rows, cols).nparts : 0;
  return cudaSuccess;
}

cudaError_t launch_ln_backward(NormRowsParams& p, int dtype, cudaStream_t st) {
  const size_t es = dtype == XP_F32 ? 4 : 2;
  const BackwardShape s = backward_shape(p.rows, p.cols);
  const bool vec = vec_rows(p.x, p.x_stride, es) && vec_rows(p.dy, p.dy_stride, es) && vec_rows(p.out, p.out_stride, es) && vec_w(p.gamma);
  cudaError_t e;
  if (dtype == XP_F32)
    e = vec ? backward<float, 4>(p, s, st) : backward<float, 1>(p, s, st);
  else
    e = vec ? backward<bf16, 8>(p, s, st) : backward<bf16, 1>(p, s, st);
  if (e != cudaSuccess || !p.dgamma || s.nparts == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(div_up(p.cols, 32), 2);
  cfg.blockDim = dim3(32 * kPartWarps);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, ln_parts_kernel, (const float*)p.partial, s.nparts, p.cols, p.dgamma, p.dbeta, p.accumulate);
}

}  // namespace xp
