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

// ---- a row's units on their way into shared memory: two at a time per thread
// (a batch), into places of its own, three batches ahead of the one in work.
constexpr int kBatch = 2, kBatches = 4;
struct Ring {
  unsigned smem, n, threads;   // this thread's first place; whole batches that it has
  const uint4* from;
  __device__ __forceinline__ Ring(const uint8_t* raw, unsigned top, const uint4* body, unsigned units) {
    threads = blockDim.x;
    smem = (unsigned)__cvta_generic_to_shared(raw) + 12 * ((top + 3) & ~3u) + 16 * threadIdx.x;
    from = body + threadIdx.x;
    const unsigned each = units > threadIdx.x ? (units - threadIdx.x - 1) / threads + 1 : 0;
    n = each / kBatch;
  }
  __device__ __forceinline__ unsigned place(unsigned b, int i) const { return smem + 16 * threads * (b % kBatches * kBatch + i); }
  __device__ __forceinline__ void bring(unsigned b) const {
    if (b < n) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(place(b, i)), "l"(from + (u64)(b * kBatch + i) * threads) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  __device__ __forceinline__ void begin() const {
#pragma unroll
    for (int b = 0; b + 1 < kBatches; ++b) bring(b);
  }
  __device__ __forceinline__ void next(unsigned b, uint4 (&q)[kBatch]) const {   // batch b, and one more on its way
    bring(b + kBatches - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kBatches - 1) : "memory");
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q[i].x), "=r"(q[i].y), "=r"(q[i].z), "=r"(q[i].w) : "r"(place(b, i)) : "memory");
  }
  // nothing lands after this
  __device__ __forceinline__ void end() const { asm volatile("cp.async.wait_group 0;" ::: "memory"); }
};

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
  float* t;
  float* z;      // the logit
};
__device__ __forceinline__ Entries entries_in(uint8_t* raw, unsigned top) {
  const unsigned room = (top + 3) & ~3u;
  return {reinterpret_cast<int*>(raw), reinterpret_cast<float*>(raw) + room, reinterpret_cast<float*>(raw) + 2 * room};
}

// Brings them.  False, the same for the CTA, if the row has none.  max_t: the
// largest of this thread's.  (The threads' first loads of the row's logits are on
// their way meanwhile: 8192 x 32000 bf16 forward 117 us without.)
template <typename T>
__device__ __forceinline__ bool bring_entries(const DistillParams& p, u64 row, const T* logits, const Entries& e, float& max_t) {
  max_t = -INFINITY;
  bool any = false;
  if (threadIdx.x < ((p.top + 3) & ~3u) - p.top) e.id[p.top + threadIdx.x] = -1;   // what fills the last four
  for (unsigned j = threadIdx.x; j < p.top; j += blockDim.x) {
    int id = p.ids[row * p.top + j];
    const float t = p.teacher[row * p.top + j];
    if ((unsigned)id >= p.vocab || t == -INFINITY) id = -1;
    e.id[j] = id;
    e.t[j] = t;
    if (id >= 0) {
      e.z[j] = to_f(logits[id]);
      max_t = fmaxf(max_t, t);
      any = true;
    }
  }
  return __syncthreads_or(any);
}

// A thread's share of a row: the running maximum m of z and the sum s of
// 2^((z - m) c).  (Differences first: z c and m c by themselves overflow where a
// mask is the type's lowest value.)  m is -infinity and s 0 while nothing above
// -infinity was met; differences are from 0 then.
struct Running {
  float m, s;
};
__device__ __forceinline__ float from(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ void raise_to(Running& r, float top, float c) {
  if (top > r.m) {
    r.s *= pow2((r.m - top) * c);   // 2^-infinity is 0
    r.m = top;
  }
}
// Two sums at once: packed additions, half the instructions.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n.reg .b64 x, y, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nadd.rn.f32x2 z, x, y;\nmov.b64 {%0, %1}, z;\n}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float b) {
  float2 d;
  asm("{\n.reg .b64 x, y;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %4};\nmul.rn.f32x2 x, x, y;\nmov.b64 {%0, %1}, x;\n}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b));
  return d;
}
// N units of 16 bytes
template <typename T, int N>
__device__ __forceinline__ void take(Running& r, const uint4 (&q)[N], float c) {
  float top = -INFINITY;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float f[4];
      unpack<T>(q[i], f);
      top = fmaxf(top, fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])));
    }
  } else {   // pairs as they are
    __nv_bfloat162 most = *reinterpret_cast<const __nv_bfloat162*>(&q[0].x);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const unsigned w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) most = __hmax2(most, *reinterpret_cast<const __nv_bfloat162*>(&w[j]));
    }
    top = fmaxf(__low2float(most), __high2float(most));
  }
  raise_to(r, top, c);
  const float low = -from(r.m);
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float f[kUnit<T>];
    unpack<T>(q[i], f);
#pragma unroll
    for (int j = 0; j < kUnit<T>; j += 2) {
      const float2 x = mul2(add2(make_float2(f[j], f[j + 1]), make_float2(low, low)), c);
      s = add2(s, make_float2(pow2(x.x), pow2(x.y)));
    }
  }
  r.s += s.x + s.y;
}
// What two threads, or warps, have, as one: the same for both.
__device__ __forceinline__ Running joined(const Running& a, float m, float s, float c) {
  const float most = fmaxf(a.m, m), low = from(most);
  return {most, a.s * pow2((a.m - low) * c) + s * pow2((m - low) * c)};
}
__device__ __forceinline__ Running warp_joined(Running r, float c) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) r = joined(r, __shfl_xor_sync(0xffffffffu, r.m, o), __shfl_xor_sync(0xffffffffu, r.s, o), c);
  return r;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
__global__ void __launch_bounds__(1024) forward_kernel(const DistillParams p) {
  constexpr int V = kUnit<T>;
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ Running words[32];
  wait_for_predecessors();
  let_successor_start();
  const Entries e = entries_in(raw, p.top);
  const u64 row = blockIdx.x;
  const T* z = static_cast<const T*>(p.logits) + row * p.logits_stride;
  const float inv_t = 1.f / p.temperature, c = inv_t * kLog2e;
  const unsigned head = head_of(z, p.vocab), units = (p.vocab - head) / V, tail = head + units * V, n = blockDim.x;
  const uint4* body = reinterpret_cast<const uint4*>(z + head);
  const Ring ring(raw, p.top, body, units);
  ring.begin();
  float max_t;
  if (!bring_entries(p, row, z, e, max_t)) {
    ring.end();
    if (threadIdx.x == 0) {
      p.loss[row] = 0.f;
      if (p.lse) p.lse[row] = 0.f;
    }
    return;
  }
  Running r = {-INFINITY, 0.f};
  for (unsigned b = 0; b < ring.n; ++b) {
    uint4 q[kBatch];
    ring.next(b, q);
    take<T>(r, q, c);
  }
  for (unsigned k = threadIdx.x + ring.n * kBatch * n; k < units; k += n) {
    const uint4 one[1] = {body[k]};
    take<T>(r, one, c);
  }
  // the row's ends: fewer elements than threads
  if (threadIdx.x < head || tail + threadIdx.x - head < p.vocab) {
    const float f = to_f(z[threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head]);
    raise_to(r, f, c);
    r.s += pow2((f - from(r.m)) * c);
  }
  r = warp_joined(r, c);
  if ((threadIdx.x & 31) == 0) words[threadIdx.x >> 5] = r;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  // the first warp: all warps' sums, then the few entries
  const unsigned nw = blockDim.x >> 5, lane = threadIdx.x;
  r = lane < nw ? words[lane] : Running{-INFINITY, 0.f};
  r = warp_joined(r, c);
  const float lse = r.m * inv_t + logf(r.s);
  float top_t = -INFINITY;
  for (unsigned j = lane; j < p.top; j += 32)
    if (e.id[j] >= 0) top_t = fmaxf(top_t, e.t[j]);
  top_t = warp_max(top_t);
  float w = 0.f;   // (differences first, as for the row)
  for (unsigned j = lane; j < p.top; j += 32)
    if (e.id[j] >= 0) w += pow2((e.t[j] - top_t) * c);
  w = warp_sum(w);
  const float log_w = logf(w);
  float loss = 0.f;
  for (unsigned j = lane; j < p.top; j += 32) {
    if (e.id[j] < 0) continue;
    const float d = e.t[j] - top_t, prob = pow2(d * c) / w;
    if (!(prob == 0.f)) loss += prob * ((d * inv_t - log_w) - (e.z[j] * inv_t - lse));
  }
  loss = warp_sum(loss);
  if (lane == 0) {
    p.loss[row] = loss * p.temperature * p.temperature;
    if (p.lse) p.lse[row] = lse;
  }
}

template <typename T>
__global__ void __launch_bounds__(1024) backward_kernel(const DistillParams p) {
  constexpr int V = kUnit<T>;
  extern __shared__ __align__(16) uint8_t raw[];
  __shared__ float words[32];
  wait_for_predecessors();
  let_successor_start();
  const Entries e = entries_in(raw, p.top);
  const u64 row = blockIdx.x;
  const T* z = static_cast<const T*>(p.logits) + row * p.logits_stride;
  T* out = static_cast<T*>(p.dlogits) + row * p.dlogits_stride;
  const float inv_t = 1.f / p.temperature, c = inv_t * kLog2e;
  const unsigned head = head_of(out, p.vocab), units = (p.vocab - head) / V, tail = head + units * V, n = blockDim.x;
  const bool alike = head_of(z, p.vocab) == head;   // z has the same phase
  const uint4* body = reinterpret_cast<const uint4*>(z + head);
  uint4* to = reinterpret_cast<uint4*>(out + head);
  const Ring ring(raw, p.top, body, alike ? units : 0);
  ring.begin();
  float max_t;
  const bool any = bring_entries(p, row, z, e, max_t);
  const float lse = any ? p.lse[row] : 0.f, scale = any ? p.dloss[row] * p.temperature : 0.f;
  // q = e^(z / T - lse); rows without entries do not look at z
  auto q_of = [&](float v) { return pow2(fmaf(v, inv_t, -lse) * kLog2e); };
  auto gradient = [&](uint4 unit) {
    float f[V];
    unpack<T>(unit, f);
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = q_of(f[j]) * scale;
    return pack<T>(f);
  };
  if (!any) {
    ring.end();
    for (unsigned k = threadIdx.x; k < units; k += n) to[k] = make_uint4(0, 0, 0, 0);
  } else if (alike) {
    for (unsigned b = 0; b < ring.n; ++b) {
      uint4 q[kBatch];
      ring.next(b, q);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) to[threadIdx.x + (b * kBatch + i) * n] = gradient(q[i]);
    }
    for (unsigned k = threadIdx.x + ring.n * kBatch * n; k < units; k += n) to[k] = gradient(body[k]);
  } else {
    for (unsigned k = threadIdx.x; k < units * V; k += blockDim.x) from_f(q_of(to_f(z[head + k])) * scale, out[head + k]);
  }
  if (threadIdx.x < head || tail + threadIdx.x - head < p.vocab) {
    const unsigned at = threadIdx.x < head ? threadIdx.x : tail + threadIdx.x - head;
    from_f(any ? q_of(to_f(z[at])) * scale : 0.f, out[at]);
  }
  if (!any) return;
  // the entries' own elements once more, with their p
  const float top_t = cta_max(max_t, words);
  float w = 0.f;
  for (unsigned j = threadIdx.x; j < p.top; j += blockDim.x)
    if (e.id[j] >= 0) w += pow2((e.t[j] - top_t) * c);
  w = cta_sum(w, words);
  for (unsigned j = threadIdx.x; j < p.top; j += blockDim.x) {
    const int id = e.id[j];
    if (id < 0) continue;
    // Mostly one entry names a token.  (Its p among the comparisons, where each lane meets itself at another step: 13558 x
    // 3001 bf16 with 115 entries 91 us, 57 so.)
    int named = 0;
    for (unsigned i = 0; i < p.top; i += 4) {
      const int4 four = *reinterpret_cast<const int4*>(e.id + i);
      named += (four.x == id) + (four.y == id) + (four.z == id) + (four.w == id);
    }
    float prob = 0.f;
    if (named == 1) {
      prob = pow2((e.t[j] - top_t) * c) / w;
    } else {   // of all entries that name it, in their order
#pragma unroll 1
      for (unsigned i = 0; i < p.top; ++i)
        if (e.id[i] == id) prob += pow2((e.t[i] - top_t) * c) / w;
    }
    from_f((q_of(e.z[j]) - prob) * scale, out[id]);
  }
}

// Threads of a row: a dozen units each (13558 x 3001 fp32 forward: 85 us with
// three), more where rows do not fill the SMs, and all that an SM has where
// there are fewer rows than SMs.  Many short rows have a warp each (16000 x 1024
// bf16 forward 19 us, 24 by two).
int threads_for(const DistillParams& p, int unit, int sms) {
  const unsigned units = (p.vocab + unit - 1) / unit;
  const unsigned most = p.rows <= (unsigned)sms ? 1024 : 256;
  unsigned n = units <= 128 && (unsigned long long)p.rows * 32 >= 1024ull * sms ? 32 : 64;
  while (n < most && n * 4 < units && (n * 12 < units || (unsigned long long)p.rows * n < 1024ull * sms)) n *= 2;
  return (int)n;
}
size_t smem_for(const DistillParams& p, int threads) { return (size_t)12 * ((p.top + 3) & ~3u) + (size_t)16 * kBatch * kBatches * threads; }

}  // namespace

cudaError_t launch_distill_forward(const DistillParams& p, int dtype, int sms, cudaStream_t st) {
  const int threads = threads_for(p, dtype == XP_F32 ? 4 : 8, sms);
  return launch_dependent(dtype == XP_F32 ? forward_kernel<float> : forward_kernel<bf16>, dim3(p.rows), threads, smem_for(p, threads), 1, st, p);
}
cudaError_t launch_distill_backward(const DistillParams& p, int dtype, int sms, cudaStream_t st) {
  const int threads = threads_for(p, dtype == XP_F32 ? 4 : 8, sms);
  return launch_dependent(dtype == XP_F32 ? backward_kernel<float> : backward_kernel<bf16>, dim3(p.rows), threads, smem_for(p, threads), 1, st, p);
}

}  // namespace xp
