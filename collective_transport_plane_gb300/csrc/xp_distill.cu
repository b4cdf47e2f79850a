// Distillation from a teacher's top logits, and its gradient
// (include/xp_model.h).
//
// The logits are by far the most that is read: once forward, with the running
// maximum and sum of the softmax, and once backward, where the gradient is
// written.  HBM bounds both, with the exponentials (one per logit) next.  A row
// belongs to a CTA; the teacher's few entries go through its shared memory.
#include "xp_model_internal.h"
#include "xp_train_device.cuh"

namespace xp {
namespace {

typedef __nv_bfloat16 bf16;
typedef unsigned long long u64;

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float v, float& x) { x = v; }
__device__ __forceinline__ void from_f(float v, bf16& x) { x = __float2bfloat16_rn(v); }
__device__ __forceinline__ unsigned pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const unsigned*>(&h);
}
// 2^x, results below 2^-126 zero
__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
constexpr int kUnit = 16 / (int)sizeof(T);

template <typename T>
__device__ __forceinline__ void unpack(uint4 q, float (&f)[kUnit<T>]) {
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
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&f)[kUnit<T>]) {
  if constexpr (sizeof(T) == 4)
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  else
    return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
}

// Elements before a row's first 16-byte boundary, at most n.
template <typename T>
__device__ __forceinline__ unsigned head_of(const T* row, unsigned n) {
  return min(n, (unsigned)((16u - (unsigned)(reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / (unsigned)sizeof(T));
}

// The CTA's maximum and sum, the same in every thread.  (A NaN is a sum's to
// carry on: fmaxf leaves it out.)
__device__ __forceinline__ float cta_max(float v, float* words) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) words[threadIdx.x >> 5] = v;
  __syncthreads();
  v = words[0];
  for (unsigned i = 1; i < blockDim.x >> 5; ++i) v = fmaxf(v, words[i]);
  return v;
}
__device__ __forceinline__ float cta_sum(float v, float* words) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) words[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (unsigned i = 0; i < blockDim.x >> 5; ++i) v += words[i];
  return v;
}

// The row's entries, laid out in shared memory.
struct Entries {
  int* id;       // -1: counts for nothing
  float* u;      // t / T
  float* z;      // the logit
};
__device__ __forceinline__ Entries entries_in(uint8_t* raw, unsigned top) {
  const unsigned room = (top + 3) & ~3u;
  return {reinterpret_cast<int*>(raw), reinterpret_cast<float*>(raw) + room, reinterpret_cast<float*>(raw) + 2 * room};
}

// Brings them.  False, the same for the CTA, if the row has none.  max_u: the
// largest of this thread's.
template <typename T>
__device__ __forceinline__ bool bring_entries(const DistillParams& p, u64 row, const T* logits, const Entries& e, float inv_t, float& max_u) {
  max_u = -INFINITY;
  bool any = false;
  for (unsigned j = threadIdx.x; j < p.top; j += blockDim.x) {
    int id = p.ids[row * p.top + j];
    const float t = p.teacher[row * p.top + j];
    if ((unsigned)id >= p.vocab || t == -INFINITY) id = -1;
    e.id[j] = id;
    e.u[j] = t * inv_t;
    if (id >= 0) {
      e.z[j] = to_f(logits[id]);
      max_u = fmaxf(max_u, t * inv_t);
      any = true;
    }
  }
  return __syncthreads_or(any);
}

// A thread's share of a row: the running maximum m and the sum s of
// 2^((z - m) c).  m is the largest z met, or -infinity, where s is 0.
struct Running {
  float m, s;
};
template <int N>
__device__ __forceinline__ void take(Running& r, const float (&f)[N], float c) {
  float top = f[0];
#pragma unroll
  for (int i = 1; i < N; ++i) top = fmaxf(top, f[i]);
  if (top > r.m) {
    r.s *= pow2((r.m - top) * c);   // 2^-infinity: 0
    r.m = top;
  }
  // nothing but -infinity (or NaN, which goes on) so far: no difference from it is formed
  const float m = r.m == -INFINITY ? 0.f : r.m;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) s += pow2((f[i] - m) * c);
  r.s += s;
}

template <typename T>
__global__ void __launch_bounds__(1024) forward_kernel(const DistillParams p) {
  constexpr int V = kUnit<T>, kAtOnce = 4;
  extern __shared__ uint8_t raw[];
  __shared__ float words[32];
  wait_for_predecessors();
  let_successor_start();
  const Entries e = entries_in(raw, p.top);
  const u64 row = blockIdx.x;
  const T* z = static_cast<const T*>(p.logits) + row * p.logits_stride;
  const float inv_t = 1.f / p.temperature, c = inv_t * kLog2e;
  float max_u;
  if (!bring_entries(p, row, z, e, inv_t, max_u)) {
    if (threadIdx.x == 0) {
      p.loss[row] = 0.f;
      if (p.lse) p.lse[row] = 0.f;
    }
    return;
  }
  Running r = {-INFINITY, 0.f};
  const unsigned head = head_of(z, p.vocab), units = (p.vocab - head) / V, tail = head + units * V;
  const uint4* body = reinterpret_cast<const uint4*>(z + head);
  unsigned k = threadIdx.x;
  for (; k + (kAtOnce - 1) * blockDim.x < units; k += kAtOnce * blockDim.x) {
    uint4 q[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) q[i] = body[k + i * blockDim.x];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      float f[V];
      unpack<T>(q[i], f);
      take<V>(r, f, c);
    }
  }
  for (; k < units; k += blockDim.x) {
    float f[V];
    unpack<T>(body[k], f);
    take<V>(r, f, c);
  }
  // the row's ends: fewer elements than threads
  if (threadIdx.x < head || tail + threadIdx.x - head < p.vocab) {
    const float f[1] = {to_f(z[threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head])};
    take<1>(r, f, c);
  }
  const float m = cta_max(r.m, words), m0 = m == -INFINITY ? 0.f : m;
  const float s = cta_sum(r.m == -INFINITY ? r.s : r.s * pow2((r.m - m0) * c), words);
  const float lse = m * inv_t + logf(s);

  const float top_u = cta_max(max_u, words);
  float w = 0.f;
  for (unsigned j = threadIdx.x; j < p.top; j += blockDim.x)
    if (e.id[j] >= 0) w += pow2((e.u[j] - top_u) * kLog2e);
  w = cta_sum(w, words);
  const float log_w = logf(w);
  float loss = 0.f;
  for (unsigned j = threadIdx.x; j < p.top; j += blockDim.x) {
    if (e.id[j] < 0) continue;
    const float d = e.u[j] - top_u, prob = pow2(d * kLog2e) / w;
    if (!(prob == 0.f)) loss += prob * ((d - log_w) - (e.z[j] * inv_t - lse));
  }
  loss = cta_sum(loss, words);
  if (threadIdx.x == 0) {
    p.loss[row] = loss * p.temperature * p.temperature;
    if (p.lse) p.lse[row] = lse;
  }
}

template <typename T>
__global__ void __launch_bounds__(1024) backward_kernel(const DistillParams p) {
  constexpr int V = kUnit<T>, kAtOnce = 4;
  extern __shared__ uint8_t raw[];
  __shared__ float words[32];
  wait_for_predecessors();
  let_successor_start();
  const Entries e = entries_in(raw, p.top);
  const u64 row = blockIdx.x;
  const T* z = static_cast<const T*>(p.logits) + row * p.logits_stride;
  T* out = static_cast<T*>(p.dlogits) + row * p.dlogits_stride;
  const float inv_t = 1.f / p.temperature, c = inv_t * kLog2e;
  float max_u;
  const bool any = bring_entries(p, row, z, e, inv_t, max_u);
  const float lse = any ? p.lse[row] : 0.f, scale = any ? p.dloss[row] * p.temperature : 0.f, lse2 = lse * kLog2e;
  // q = 2^(z c - lse2); rows without entries do not look at z
  auto q_of = [&](float v) { return pow2(fmaf(v, c, -lse2)); };
  const unsigned head = head_of(out, p.vocab), units = (p.vocab - head) / V, tail = head + units * V;
  const bool alike = head_of(z, p.vocab) == head;   // z has the same phase
  uint4* to = reinterpret_cast<uint4*>(out + head);
  if (!any) {
    for (unsigned k = threadIdx.x; k < units; k += blockDim.x) to[k] = make_uint4(0, 0, 0, 0);
  } else if (alike) {
    const uint4* body = reinterpret_cast<const uint4*>(z + head);
    unsigned k = threadIdx.x;
    for (; k + (kAtOnce - 1) * blockDim.x < units; k += kAtOnce * blockDim.x) {
      uint4 q[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) q[i] = body[k + i * blockDim.x];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        float f[V];
        unpack<T>(q[i], f);
#pragma unroll
        for (int j = 0; j < V; ++j) f[j] = q_of(f[j]) * scale;
        to[k + i * blockDim.x] = pack<T>(f);
      }
    }
    for (; k < units; k += blockDim.x) {
      float f[V];
      unpack<T>(body[k], f);
#pragma unroll
      for (int j = 0; j < V; ++j) f[j] = q_of(f[j]) * scale;
      to[k] = pack<T>(f);
    }
  } else {
    for (unsigned k = threadIdx.x; k < units * V; k += blockDim.x) from_f(q_of(to_f(z[head + k])) * scale, out[head + k]);
  }
  if (threadIdx.x < head || tail + threadIdx.x - head < p.vocab) {
    const unsigned at = threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;
    from_f(any ? q_of(to_f(z[at])) * scale : 0.f, out[at]);
  }
  if (!any) return;
  // the entries' own elements once more, with their p
  const float top_u = cta_max(max_u, words);
  float w = 0.f;
  for (unsigned j = threadIdx.x; j < p.top; j += blockDim.x)
    if (e.id[j] >= 0) w += pow2((e.u[j] - top_u) * kLog2e);
  w = cta_sum(w, words);
  for (unsigned j = threadIdx.x; j < p.top; j += blockDim.x) {
    const int id = e.id[j];
    if (id < 0) continue;
    float prob = 0.f;   // of all entries that name the token, in their order
    for (unsigned i = 0; i < p.top; ++i)
      if (e.id[i] == id) prob += pow2((e.u[i] - top_u) * kLog2e) / w;
    from_f((q_of(e.z[j]) - prob) * scale, out[id]);
  }
}

// Threads of a row: all the SM has where rows are few, else enough for the
// row's units, four at a time.
int threads_for(const DistillParams& p, int unit, int sms) {
  const unsigned units = (p.vocab + unit - 1) / unit;
  const unsigned most = p.rows <= (unsigned)sms ? 1024 : 256;
  unsigned n = 64;
  while (n < most && n * 4 < units) n *= 2;
  return (int)n;
}
size_t smem_for(const DistillParams& p) { return (size_t)3 * ((p.top + 3) & ~3u) * 4; }

}  // namespace

cudaError_t launch_distill_forward(const DistillParams& p, int dtype, int sms, cudaStream_t st) {
  if (dtype == XP_F32) return launch_dependent(forward_kernel<float>, dim3(p.rows), threads_for(p, 4, sms), smem_for(p), 1, st, p);
  return launch_dependent(forward_kernel<bf16>, dim3(p.rows), threads_for(p, 8, sms), smem_for(p), 1, st, p);
}
cudaError_t launch_distill_backward(const DistillParams& p, int dtype, int sms, cudaStream_t st) {
  if (dtype == XP_F32) return launch_dependent(backward_kernel<float>, dim3(p.rows), threads_for(p, 4, sms), smem_for(p), 1, st, p);
  return launch_dependent(backward_kernel<bf16>, dim3(p.rows), threads_for(p, 8, sms), smem_for(p), 1, st, p);
}

}  // namespace xp
