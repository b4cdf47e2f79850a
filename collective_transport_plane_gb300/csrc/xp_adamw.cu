// AdamW over many tensors at once, the global gradient norm before it, and
// the values of 8-bit states.  include/xp_train.h states the formulas.
//
// All three are elementwise or a sum: what bounds them is the memory they
// move.  A group's tensors are cut into units once, at creation, and one
// launch covers every tensor, so many small tensors cost no more launches
// than one.
#include "xp_train_device.cuh"

namespace xp {
namespace {

// ---------------------------------------------------------------- vectors of kVec elements

template <typename T>
struct Raw;
template <>
struct Raw<float> {
  uint4 q[2];
};
template <>
struct Raw<__nv_bfloat16> {
  uint4 q[1];
};

template <typename T>
__device__ __forceinline__ Raw<T> load_vec(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(Raw<T>) / 16); ++i) r.q[i] = reinterpret_cast<const uint4*>(p)[i];
  return r;
}
__device__ __forceinline__ void widen(const Raw<float>& r, float (&f)[kVec]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    f[4 * i] = __uint_as_float(r.q[i].x);
    f[4 * i + 1] = __uint_as_float(r.q[i].y);
    f[4 * i + 2] = __uint_as_float(r.q[i].z);
    f[4 * i + 3] = __uint_as_float(r.q[i].w);
  }
}
__device__ __forceinline__ void widen(const Raw<__nv_bfloat16>& r, float (&f)[kVec]) {
  const unsigned w[4] = {r.q[0].x, r.q[0].y, r.q[0].z, r.q[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store_vec(float* p, const float (&f)[kVec]) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(f[4 * i], f[4 * i + 1], f[4 * i + 2], f[4 * i + 3]);
}
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&f)[kVec]) {
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<uint4*>(h);
}
__device__ __forceinline__ float one(const float* p) { return *p; }
__device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void put(float* p, float f) { *p = f; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float f) { *p = __float2bfloat16_rn(f); }

// n of kVec elements at p (n < kVec at a tensor's end, and at any n where the
// pointer allows no vector); the rest read as 0.
template <typename T>
__device__ __forceinline__ void load_some(const T* p, int n, bool vec, float (&f)[kVec]) {
  if (vec && n == kVec) {
    widen(load_vec(p), f);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[i] = i < n ? one(p + i) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void store_some(T* p, int n, bool vec, const float (&f)[kVec]) {
  if (vec && n == kVec) {
    store_vec(p, f);
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      if (i < n) put(p + i, f[i]);
  }
}
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int n, bool vec) {
  if (vec && n == kVec) return *reinterpret_cast<const uint2*>(p);
  uint2 c = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < kVec; ++i)
    if (i < n) (i < 4 ? c.x : c.y) |= (unsigned)p[i] << (8 * (i & 3));
  return c;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int n, bool vec, uint2 c) {
  if (vec && n == kVec) {
    *reinterpret_cast<uint2*>(p) = c;
    return;
  }
#pragma unroll
  for (int i = 0; i < kVec; ++i)
    if (i < n) p[i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
}
// Whether kVec elements of T starting at a multiple of kVec may move at once.
template <typename T>
__device__ __forceinline__ bool vec_ok(const T* p) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

// ---------------------------------------------------------------- 8-bit states

// The fp32 pattern's last 20 bits are cut: what is left is the exponent and 3
// mantissa bits, a whole number that the block's exponent shifts into 7 or 8
// bits.  Decoding and encoding are integer operations on it, exact, with no
// division by the block's scale.
template <bool SIGNED>
constexpr int kShift = SIGNED ? 119 : 247;

template <bool SIGNED>
__device__ __forceinline__ void decode_codes(uint2 c, int e, float (&f)[kVec]) {
  const int base = 8 * e - kShift<SIGNED>;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const int b = (int)(((i < 4 ? c.x : c.y) >> (8 * (i & 3))) & 0xffu);
    const int mag = SIGNED ? (b & 127) : b;
    unsigned bits = (unsigned)max(mag + base, 0) << 20;
    bits = mag == 0 ? 0u : bits;
    if (SIGNED) bits |= (unsigned)(b & 128) << 24;
    f[i] = e == 255 ? __uint_as_float(0x7fc00000u) : __uint_as_float(bits);
  }
}

// exponent of the largest magnitude among a thread's elements
__device__ __forceinline__ unsigned top_exponent(const float (&f)[kVec]) {
  unsigned top = 0;
#pragma unroll
  for (int i = 0; i < kVec; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
  return top >> 23;
}

template <bool SIGNED>
__device__ __forceinline__ unsigned encode_one(float x, unsigned noise, int e) {
  const unsigned bits = __float_as_uint(x) & 0x7fffffffu;
  int c = (int)((bits + noise) >> 20) - (8 * e - kShift<SIGNED>);
  c = min(max(c, SIGNED ? 0 : 1), SIGNED ? 127 : 255);
  c = bits == 0 ? 0 : c;
  if (SIGNED && c > 0) c |= (int)(__float_as_uint(x) >> 24) & 128;
  return (unsigned)c;
}

// Two products at once, and two sums one by one: a product that feeds a sum
// must be rounded by itself, and a packed product before a packed sum is fused
// into one operation whatever the flags (seen as 1 ulp of the weights).
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float b) { return __fmul2_rn(a, make_float2(b, b)); }
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y)); }

// The same for a thread's eight elements, in fewer operations; the results are
// the same bits.
//
// Decoding: a code's fp32 pattern has nothing below its upper half, which is
// (magnitude + base) << 4: two codes go in one register, as a pair of bf16.
// em and ev >= 32, or all codes 0; finite.
__device__ __forceinline__ bool pairs_ok(uint2 c, int e) { return (e >= 32 || (c.x | c.y) == 0) && e != 255; }
template <bool SIGNED>
__device__ __forceinline__ void decode_pairs(uint2 c, int e, unsigned (&w)[kVec / 2]) {
  const unsigned base = 16u * (unsigned)max(8 * e - kShift<SIGNED>, 0);
#pragma unroll
  for (int i = 0; i < kVec / 2; ++i) {
    const unsigned x = __byte_perm(i < 2 ? c.x : c.y, 0, i & 1 ? 0x4342u : 0x4140u);
    const unsigned mag = SIGNED ? x & 0x007f007fu : x;
    w[i] = mag * 16u + __vminu2(mag, 0x00010001u) * base;   // 0 for magnitude 0
    if (SIGNED) w[i] |= (x << 8) & 0x80008000u;
  }
}
__device__ __forceinline__ void widen_pairs(const unsigned (&w)[kVec / 2], float2 (&f)[kVec / 2]) {
#pragma unroll
  for (int i = 0; i < kVec / 2; ++i) f[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

// Encoding: z = pattern + noise - (base << 20) has the code in bits 20 to 27;
// shifted to the top byte, four of them are gathered by byte permutations.
// em >= 16 and ev >= 32 (so that 0 gives 0).
struct Encoder {
  int cm, cv;
  uint2 m, v;
  unsigned zm[4], zv[4];
  __device__ __forceinline__ Encoder(int em, int ev)
      : cm(8 - ((8 * em - kShift<true>) << 20)), cv(8 - ((8 * ev - kShift<false>) << 20)) {}
  // element k: m's pattern, v's pattern, the hashes in two registers
  __device__ __forceinline__ void put(int k, unsigned bm, unsigned bv, unsigned hm, unsigned hv) {
    const int a = __viaddmax_s32((int)(hm * 16u + (bm & 0x7fffffffu)), cm, 0);
    const int b = __viaddmax_s32((int)(hv * 16u + bv), cv, (int)(min(bv, 1u) << 20));   // a positive v keeps code 1
    zm[k & 3] = ((unsigned)a << 4) | (bm & 0x80000000u);
    zv[k & 3] = (unsigned)b << 4;
    if ((k & 3) == 3) {
      unsigned c = __byte_perm(__byte_perm(zm[0], zm[1], 0x0073), __byte_perm(zm[2], zm[3], 0x0073), 0x5410);
      c &= ((c & 0x7f7f7f7fu) + 0x7f7f7f7fu) | 0x7f7f7f7fu;   // no sign without a magnitude
      const unsigned d = __byte_perm(__byte_perm(zv[0], zv[1], 0x0073), __byte_perm(zv[2], zv[3], 0x0073), 0x5410);
      (k < 4 ? m.x : m.y) = c;
      (k < 4 ? v.x : v.y) = d;
    }
  }
};

// A 32-bit mix of the step and the position: multiplications by odd constants
// and shifts, each invertible, so that positions never collide within a key.
__device__ __forceinline__ unsigned mix_last(unsigned x) {   // but for its last xor
  x = (x ^ (x >> 16)) * 0xDDF15BA9u;
  return (x ^ (x >> 15)) * 0xE31B8755u;
}
__device__ __forceinline__ unsigned mix(unsigned x) {
  x = mix_last(x);
  return x ^ (x >> 16);
}
constexpr unsigned kPosLo = 0x8ED88009u, kPosHi = 0xB86D3E2Fu;
__device__ __forceinline__ unsigned step_key(unsigned seed, unsigned step) { return mix(seed * kPosLo + mix(step)); }

// Square roots and quotients, two at a time and without the range checks and
// branches of the functions' own: Markstein's iterations (P. W. Markstein,
// "Computation of elementary functions on the IBM RISC System/6000
// processor", IBM Journal of Research and Development 34, 1990), in which
// fused multiply-adds give exact remainders.  Correctly rounded where neither
// results nor remainders leave fp32's normal range, as the caller sees to.  (A
// remainder is a multiple of 2^-46 of its numerator at least.)
__device__ __forceinline__ float2 both(float a) { return make_float2(a, a); }
__device__ __forceinline__ float approximate_rsqrt(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float approximate_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Signs are changed by exact products, which are packed too.
__device__ __forceinline__ float2 root2(float2 v) {
  const float2 y = make_float2(approximate_rsqrt(v.x), approximate_rsqrt(v.y));
  float2 g = mul2(v, y), h = mul2(y, -0.5f);
  const float2 r = __ffma2_rn(h, g, both(0.5f));
  g = __ffma2_rn(g, r, g);
  h = __ffma2_rn(h, r, h);
  return __ffma2_rn(h, __ffma2_rn(g, g, mul2(v, -1.f)), g);
}
__device__ __forceinline__ float2 quotient2(float2 a, float2 d) {
  float2 y = make_float2(approximate_rcp(d.x), approximate_rcp(d.y));
  d = mul2(d, -1.f);
  y = __ffma2_rn(y, __ffma2_rn(d, y, both(1.f)), y);
  const float2 q = mul2(a, y);
  return __ffma2_rn(__ffma2_rn(d, q, a), y, q);
}

// Where a thread's eight elements with 8-bit states are, and what they take
// from memory.
template <typename P, typename G>
struct Place8 {
  P* param;
  const G* grad;
  uint8_t *m, *v, *m_scale, *v_scale;
  __nv_bfloat16* copy;
  __device__ __forceinline__ Place8(const GroupTensor& t, unsigned long long i)
      : param(static_cast<P*>(t.param) + i), grad(static_cast<const G*>(t.grad) + i), m(static_cast<uint8_t*>(t.m) + i),
        v(static_cast<uint8_t*>(t.v) + i), m_scale(t.m_scale + i / XP_STATE8_BLOCK), v_scale(t.v_scale + i / XP_STATE8_BLOCK),
        copy(t.copy ? static_cast<__nv_bfloat16*>(t.copy) + i : nullptr) {}
  __device__ __forceinline__ void advance(int n) {
    param += n, grad += n, m += n, v += n;
    m_scale += n / XP_STATE8_BLOCK, v_scale += n / XP_STATE8_BLOCK;
    if (copy) copy += n;
  }
};
template <typename P, typename G>
struct Values8 {
  Raw<G> g;
  Raw<P> p;
  uint2 cm, cv;
  int em, ev;
  __device__ __forceinline__ void load(const Place8<P, G>& at, int ahead) {
    g = load_vec(at.grad + ahead);
    p = load_vec(at.param + ahead);
    cm = *reinterpret_cast<const uint2*>(at.m + ahead);
    cv = *reinterpret_cast<const uint2*>(at.v + ahead);
    em = at.m_scale[ahead / XP_STATE8_BLOCK];
    ev = at.v_scale[ahead / XP_STATE8_BLOCK];
  }
};

// One unit per CTA, kVec elements per thread at a time.  One thread keeps the
// books: it reads the words that live from step to step for its CTA, counts it
// in, and in the CTA that was counted last writes the next step's words, as
// all have read these.  With fp32 states it is in a warp of its own, beside
// the work (a step of 5000 elements: 4.0 us, and 5.6 with thread 0 keeping the
// books at the end); with 8-bit states, where registers are short, thread 0.
template <bool S8>
constexpr int kBooksThreads = S8 ? 0 : 32;
template <typename P, typename G, bool S8>
__global__ void __launch_bounds__(kStepThreads + kBooksThreads<S8>, 3) adamw_kernel(const __grid_constant__ StepParams prm) {
  __shared__ float s_coef[2];
  __shared__ unsigned s_step;
  const GroupUnit u = prm.units[blockIdx.x];   // never written after the group's creation
  wait_for_predecessors();
  let_successor_start();
  if (prm.report && prm.skip_nonfinite && prm.report->nonfinite) return;   // the same answer in every CTA
  unsigned arrived = 0;
  unsigned long long step = 0;
  double power1 = 0.0, power2 = 0.0;
  auto read_words = [&] {
    const volatile GroupState* st = prm.state;
    step = st->step;
    if (!S8) power1 = st->power1, power2 = st->power2;
    s_coef[0] = st->inv_bias1;
    s_coef[1] = st->inv_sqrt_bias2;
    s_step = (unsigned)(step + 1);
  };
  auto count_in = [&] {
    __threadfence();
    arrived = atomicAdd(&prm.state->arrived_step, 1u) + 1;
  };
  auto next_words = [&] {
    if (arrived != gridDim.x) return;
    GroupState* st = prm.state;
    if (S8) power1 = st->power1, power2 = st->power2;   // not held through the work
    const double n1 = power1 * prm.beta1_d, n2 = power2 * prm.beta2_d;
    st->step = step + 1;
    st->power1 = n1;
    st->power2 = n2;
    st->inv_bias1 = (float)(1.0 / (1.0 - n1));
    st->inv_sqrt_bias2 = (float)(1.0 / sqrt(1.0 - n2));
    st->arrived_step = 0;
  };
  if (!S8 && threadIdx.x >= kStepThreads) {
    if (threadIdx.x == kStepThreads) read_words();
    __syncthreads();
    if (threadIdx.x == kStepThreads) {
      count_in();
      next_words();
    }
    return;
  }
  if (S8 && threadIdx.x == 0) read_words();
  const GroupTensor t = prm.tensors[u.tensor];
  const float lr = prm.lr_dev ? *prm.lr_dev : prm.lr;
  const float gscale = prm.report ? prm.report->scale : prm.grad_scale;
  const float keep = 1.0f - lr * t.decay;
  P* param = static_cast<P*>(t.param) + u.start;
  const G* grad = static_cast<const G*>(t.grad) + u.start;
  const bool vec = t.aligned && vec_ok(static_cast<const G*>(t.grad));

  // every thread of a warp makes the same number of turns: 8-bit blocks
  // share their exponent by shuffles
  constexpr unsigned kTurn = kStepThreads * kVec;
  const unsigned turns = (u.n + kTurn - 1) / kTurn;
  float alpha = 0.f, rs = 0.f;
  unsigned key = 0;
  unsigned top_v = 0, least_m = 0;   // patterns between which root2 and quotient2 serve (8-bit states)
  auto coefficients = [&](unsigned turn) {   // after the first turn's loads are on their way
    if (turn) return;
    __syncthreads();
    if (S8 && threadIdx.x == 0) count_in();
    alpha = lr * s_coef[0];
    rs = s_coef[1];
    if (S8) {
      key = step_key(prm.seed, s_step);
      // with v up to 2^40 a denominator is between 2^-50 and `most`; numerators of 2^-100 and more have exact
      // remainders, and of 2^-120 `most` and more normal quotients
      const float most = 0x1p20f * rs + prm.eps;
      top_v = most <= 0x1p100f && fabsf(alpha) <= 0x1p20f ? 167u << 23 : 0u;
      least_m = alpha != 0.f ? 2u * __float_as_uint(fmaxf(0x1p-100f, 0x1p-120f * most) / fabsf(alpha)) : 0u;
    }
  };
  if (turns == 0) coefficients(0);
  unsigned turn = 0;
  const unsigned whole = vec ? u.n / kTurn : 0;   // turns of eight aligned elements for every thread
  if constexpr (S8) {
    Place8<P, G> place(t, u.start + threadIdx.x * kVec);
    unsigned long long pos = t.pos + u.start + threadIdx.x * kVec;
    Values8<P, G> next;
    if (whole > 0) next.load(place, 0);
    for (; turn < whole; ++turn, pos += kTurn) {
      const Values8<P, G> now = next;
      if (turn + 1 < whole) next.load(place, kTurn);
      coefficients(turn);
      float2 m[kVec / 2], v[kVec / 2];
      if (pairs_ok(now.cm, now.em) && pairs_ok(now.cv, now.ev)) {
        unsigned wm[kVec / 2], wv[kVec / 2];
        decode_pairs<true>(now.cm, now.em, wm);
        decode_pairs<false>(now.cv, now.ev, wv);
        widen_pairs(wm, m);
        widen_pairs(wv, v);
      } else {
        float fm[kVec], fv[kVec];
        decode_codes<true>(now.cm, now.em, fm);
        decode_codes<false>(now.cv, now.ev, fv);
#pragma unroll
        for (int k = 0; k < kVec / 2; ++k) {
          m[k] = make_float2(fm[2 * k], fm[2 * k + 1]);
          v[k] = make_float2(fv[2 * k], fv[2 * k + 1]);
        }
      }
      float g[kVec], p[kVec];
      widen(now.g, g);
      widen(now.p, p);
#pragma unroll
      for (int k = 0; k < kVec / 2; ++k) {
        const float2 gi = mul2(make_float2(g[2 * k], g[2 * k + 1]), gscale);
        m[k] = add2(mul2(m[k], prm.beta1), mul2(gi, prm.one_minus_beta1));
        v[k] = add2(mul2(v[k], prm.beta2), mul2(mul2(gi, prm.one_minus_beta2), gi));
      }
      unsigned tm = 0, tv = 0, lv = 0xffffffffu, lm = 0xffffffffu;   // largest magnitudes, smallest v, smallest m but 0 (less 1)
#pragma unroll
      for (int k = 0; k < kVec / 2; ++k) {
        const unsigned mx = __float_as_uint(m[k].x) * 2u, my = __float_as_uint(m[k].y) * 2u;   // without their signs
        tm = max(max(tm, mx), my);
        lm = __viaddmin_u32(my, 0xffffffffu, __viaddmin_u32(mx, 0xffffffffu, lm));
        tv = max(max(tv, __float_as_uint(v[k].x)), __float_as_uint(v[k].y));
        lv = min(min(lv, __float_as_uint(v[k].x)), __float_as_uint(v[k].y));
      }
      // v in [2^-100, 2^40], m up to 2^50 and above least_m or 0: roots, quotients and remainders are in range (without
      // the least m, 100 M elements take 252 us and not 258, but quotients near 0 lose bits)
      const bool in_range = lv >= 27u << 23 && tv <= top_v && tm <= 177u << 24 && lm >= least_m;
      auto weights = [&](auto root, auto quotient) {
#pragma unroll
        for (int k = 0; k < kVec / 2; ++k) {
          const float2 d = add2(mul2(root(v[k]), rs), both(prm.eps)), q = quotient(mul2(m[k], alpha), d);
          const float2 kept = mul2(make_float2(p[2 * k], p[2 * k + 1]), keep);
          p[2 * k] = __fsub_rn(kept.x, q.x);
          p[2 * k + 1] = __fsub_rn(kept.y, q.y);
        }
      };
      if (in_range)
        weights([](float2 x) { return root2(x); }, [](float2 a, float2 d) { return quotient2(a, d); });
      else
        weights([](float2 x) { return make_float2(__fsqrt_rn(x.x), __fsqrt_rn(x.y)); },
                [](float2 a, float2 d) { return make_float2(__fdiv_rn(a.x, d.x), __fdiv_rn(a.y, d.y)); });
      store_vec(place.param, p);
      if (place.copy) store_vec(place.copy, p);
      unsigned top = (tm >> 24) << 16 | (tv >> 23 & 0xffu);
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int em = (int)(top >> 16), ev = (int)(top & 0xffffu);
      uint2 cm, cv;
      unsigned h = (unsigned)pos * kPosLo + (unsigned)(pos >> 32) * kPosHi + key;   // kVec positions share the high word
      if (em >= 16 && ev >= 32) {
        Encoder enc(em, ev);
#pragma unroll
        for (int k = 0; k < kVec; ++k, h += kPosLo) {
          const unsigned r = mix_last(h);
          const float2 mk = m[k / 2], vk = v[k / 2];
          enc.put(k, __float_as_uint(k & 1 ? mk.y : mk.x), __float_as_uint(k & 1 ? vk.y : vk.x), r >> 16, (r ^ (r >> 16)) & 0xffffu);
        }
        cm = enc.m;
        cv = enc.v;
      } else {
        cm = cv = make_uint2(0, 0);
#pragma unroll
        for (int k = 0; k < kVec; ++k, h += kPosLo) {
          const unsigned r = mix(h);
          const float2 mk = m[k / 2], vk = v[k / 2];
          (k < 4 ? cm.x : cm.y) |= encode_one<true>(k & 1 ? mk.y : mk.x, ((r >> 16) << 4) + 8u, em) << (8 * (k & 3));
          (k < 4 ? cv.x : cv.y) |= encode_one<false>(k & 1 ? vk.y : vk.x, ((r & 0xffffu) << 4) + 8u, ev) << (8 * (k & 3));
        }
      }
      *reinterpret_cast<uint2*>(place.m) = cm;
      *reinterpret_cast<uint2*>(place.v) = cv;
      if ((threadIdx.x & 3) == 0) {   // a block is four threads' elements
        *place.m_scale = (uint8_t)em;
        *place.v_scale = (uint8_t)ev;
      }
      place.advance(kTurn);
    }
  }
  for (; turn < turns; ++turn) {
    const unsigned at = turn * kTurn + threadIdx.x * kVec;
    const unsigned long long i = u.start + at, pos = t.pos + i;
    uint8_t* const code_m = static_cast<uint8_t*>(t.m) + i;
    uint8_t* const code_v = static_cast<uint8_t*>(t.v) + i;
    const int n = at < u.n ? (int)min((unsigned)kVec, u.n - at) : 0;
    float p[kVec], g[kVec], m[kVec], v[kVec];
    load_some(grad + at, n, vec, g);
    load_some(param + at, n, vec, p);
    if constexpr (S8) {
      decode_codes<true>(load_codes(code_m, n, vec), n ? t.m_scale[i / XP_STATE8_BLOCK] : 0, m);
      decode_codes<false>(load_codes(code_v, n, vec), n ? t.v_scale[i / XP_STATE8_BLOCK] : 0, v);
    } else {
      load_some(static_cast<const float*>(t.m) + i, n, vec, m);
      load_some(static_cast<const float*>(t.v) + i, n, vec, v);
    }
    coefficients(turn);
#pragma unroll
    for (int k = 0; k < kVec; ++k) {
      const float gi = g[k] * gscale;
      m[k] = m[k] * prm.beta1 + gi * prm.one_minus_beta1;
      v[k] = v[k] * prm.beta2 + gi * prm.one_minus_beta2 * gi;
      const float d = __fsqrt_rn(v[k]) * rs + prm.eps;
      // a numerator of 0, which weights without gradients have, would take the division's slow path, and its warp with
      // it; d > 0 or NaN, and over a NaN it is a NaN too
      const float a = m[k] * alpha;
      const bool zero = a == 0.f && d == d;
      const float q = __fdiv_rn(zero ? 1.f : a, d);
      p[k] = p[k] * keep - (zero ? a : q);
    }
    store_some(param + at, n, vec, p);
    if (t.copy) store_some(static_cast<__nv_bfloat16*>(t.copy) + i, n, vec, p);
    if constexpr (S8) {
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        if (k >= n) m[k] = v[k] = 0.f;
      unsigned top = top_exponent(m) << 16 | top_exponent(v);
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const int em = (int)(top >> 16), ev = (int)(top & 0xffffu);
      uint2 cm = make_uint2(0, 0), cv = make_uint2(0, 0);
      unsigned h = (unsigned)pos * kPosLo + (unsigned)(pos >> 32) * kPosHi + key;
#pragma unroll
      for (int k = 0; k < kVec; ++k, h += kPosLo) {
        const unsigned r = mix(h);
        (k < 4 ? cm.x : cm.y) |= encode_one<true>(m[k], ((r >> 16) << 4) + 8u, em) << (8 * (k & 3));
        (k < 4 ? cv.x : cv.y) |= encode_one<false>(v[k], ((r & 0xffffu) << 4) + 8u, ev) << (8 * (k & 3));
      }
      store_codes(code_m, n, vec, cm);
      store_codes(code_v, n, vec, cv);
      if (n && (threadIdx.x & 3) == 0) {
        t.m_scale[i / XP_STATE8_BLOCK] = (uint8_t)em;
        t.v_scale[i / XP_STATE8_BLOCK] = (uint8_t)ev;
      }
    } else {
      store_some(static_cast<float*>(t.m) + i, n, vec, m);
      store_some(static_cast<float*>(t.v) + i, n, vec, v);
    }
  }
  if (S8 && threadIdx.x == 0) next_words();
}

// ---------------------------------------------------------------- the norm

template <typename F>
__device__ __forceinline__ F warp_sum(F x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A warp's squares with sums in fp64 beyond eight elements, where its fp32 sum
// of unit `bad` became an infinity.  (Not a NaN: squares give that only where
// an element is one.)  If an element's own square is infinite there, that is the
// answer; else all units are added up again.  Not inlined, and after the loop
// over the units: what the call needs there cost the loop registers (2^27 fp32:
// 85 us, 80 so).
template <typename G>
__device__ __noinline__ double squares64(const NormParams& prm, unsigned bad) {
  double sum = 0.0;
  bool infinite = false;
  auto add_unit = [&](unsigned k) {
    const GroupUnit u = prm.units[prm.nunits - 1 - k];
    const G* grad = static_cast<const G*>(prm.tensors[u.tensor].grad);
    for (unsigned at = threadIdx.x * kVec; at < u.n; at += kNormThreads * kVec) {
      float f[kVec], eight = 0.f;
      load_some(grad + u.start + at, (int)min((unsigned)kVec, u.n - at), vec_ok(grad), f);
#pragma unroll
      for (int i = 0; i < kVec; ++i) eight += f[i] * f[i];
      if (isfinite(eight)) {
        sum += (double)eight;
        continue;
      }
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        infinite |= isinf(f[i] * f[i]);
        sum += (double)(f[i] * f[i]);
      }
    }
  };
  add_unit(bad);
  if (__any_sync(0xffffffffu, infinite)) return (double)__int_as_float(0x7f800000);
  sum = 0.0;
  for (unsigned k = blockIdx.x; k < prm.nunits; k += gridDim.x) add_unit(k);
  return warp_sum(sum);
}

// Each CTA adds up its units' squares and leaves one fp64 sum; the CTA that
// arrives last adds the sums up in their order, so the result does not depend
// on which CTA that is.  fp32 up to a warp's sum (fp64 if that overflows), fp64
// above: an SM does 2 fp64 additions per clock.  The units are taken from the last to the first, so
// that L2 holds the gradients a step reads first; the next unit's place is
// looked up while one is added.
template <typename G>
__global__ void __launch_bounds__(kNormThreads, 5) grad_norm_kernel(const __grid_constant__ NormParams prm) {
  __shared__ double s_sum[kNormThreads / 32];
  __shared__ bool s_last;
  // Where a unit whose sum became an infinity is noted: fp32 has no register to
  // spare (2^27: 82 us in one, 80 so), bf16 has (44.5 us, 47 in shared memory).
  constexpr bool kBadShared = sizeof(G) == 4;
  __shared__ unsigned s_bad[kBadShared ? kNormThreads / 32 : 1];
  constexpr unsigned kTurn = kNormThreads * kVec;
  constexpr int kDeep = sizeof(G) == 2 ? 4 : 2;   // loads of a thread in flight, 64 bytes
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned k = blockIdx.x;
  GroupUnit u = prm.units[prm.nunits - 1 - k];   // never written after the group's creation
  wait_for_predecessors();
  let_successor_start();
  const G* grad = static_cast<const G*>(prm.tensors[u.tensor].grad);
  double sum = 0.0;
  unsigned bad = 0;
  while (true) {
    const G* g = grad + u.start + threadIdx.x * kVec;
    const unsigned n = u.n, after = k + gridDim.x;
    const bool vec = vec_ok(grad), more = after < prm.nunits;
    float acc[kVec] = {};
    auto add = [&](const float (&f)[kVec]) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[i] = fmaf(f[i], f[i], acc[i]);
    };
    if (more) u = prm.units[prm.nunits - 1 - after];
    unsigned at = 0;
    if (vec) {
      for (; n - at >= kDeep * kTurn; at += kDeep * kTurn) {
        Raw<G> r[kDeep];
#pragma unroll
        for (int i = 0; i < kDeep; ++i) r[i] = load_vec(g + at + i * kTurn);
        if (more) grad = static_cast<const G*>(prm.tensors[u.tensor].grad);
#pragma unroll
        for (int i = 0; i < kDeep; ++i) {
          float f[kVec];
          widen(r[i], f);
          add(f);
        }
      }
    }
    for (; at + threadIdx.x * kVec < n; at += kTurn) {
      float f[kVec];
      load_some(g + at, (int)min((unsigned)kVec, n - at - threadIdx.x * kVec), vec, f);
      add(f);
    }
    if (more) grad = static_cast<const G*>(prm.tensors[u.tensor].grad);
    const float w = warp_sum(((acc[0] + acc[1]) + (acc[2] + acc[3])) + ((acc[4] + acc[5]) + (acc[6] + acc[7])));
    if (lane == 0) {
      sum += (double)w;
      if (kBadShared && isinf(w)) s_bad[warp] = k;
    }
    if (!kBadShared && isinf(w)) bad = k;
    if (!more) break;
    k = after;
  }
  if (__any_sync(0xffffffffu, isinf(sum))) {
    __syncwarp();
    sum = squares64<G>(prm, kBadShared ? s_bad[warp] : bad);
  }
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kNormThreads / 32; ++w) sum += s_sum[w];
    prm.partial[blockIdx.x] = sum;
    __threadfence();
    s_last = atomicAdd(&prm.state->arrived_norm, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  sum = 0.0;
  for (unsigned k = threadIdx.x; k < gridDim.x; k += kNormThreads) sum += __ldcg(prm.partial + k);
  sum = warp_sum(sum);
  __syncthreads();
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double total = prm.accumulate ? prm.report->sumsq : 0.0;
    for (int w = 0; w < kNormThreads / 32; ++w) total += s_sum[w];
    const float norm = (float)((double)prm.grad_scale * sqrt(total));
    float scale = prm.grad_scale;
    if (prm.max_norm > 0.f && norm > prm.max_norm) scale *= prm.max_norm / norm;
    prm.report->sumsq = total;
    prm.report->norm = norm;
    prm.report->scale = scale;
    prm.report->nonfinite = isfinite(total) ? 0 : 1;
    prm.state->arrived_norm = 0;
  }
}

// ---------------------------------------------------------------- small ones

__global__ void set_grads_kernel(const __grid_constant__ SetGradsParams prm) {
  wait_for_predecessors();
  let_successor_start();
  for (int i = threadIdx.x; i < prm.n; i += blockDim.x) prm.tensors[prm.first + i].grad = prm.grad[i];
}

__global__ void set_step_kernel(GroupState* s, unsigned long long step, double p1, double p2) {
  wait_for_predecessors();
  let_successor_start();
  s->step = step;
  s->power1 = p1;
  s->power2 = p2;
  s->inv_bias1 = (float)(1.0 / (1.0 - p1));
  s->inv_sqrt_bias2 = (float)(1.0 / sqrt(1.0 - p2));
  s->arrived_step = 0;
  s->arrived_norm = 0;
}

// m in the grid's row 0, v in row 1; a thread takes kVec codes at each of two places.
template <typename O>
__global__ void __launch_bounds__(kStepThreads) decode_kernel(const __grid_constant__ DecodeParams prm) {
  wait_for_predecessors();
  let_successor_start();
  const int which = blockIdx.y;
  O* out = static_cast<O*>(prm.out[which]);
  if (!out) return;
  const uint8_t* code = prm.code[which];
  const bool vec = (reinterpret_cast<uintptr_t>(code) & 7u) == 0, vec_out = vec_ok(out);
  const unsigned long long first = (unsigned long long)blockIdx.x * kDecodeCta + threadIdx.x * kVec;
  uint2 c[2];
  int e[2], n[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const unsigned long long at = first + j * (kDecodeCta / 2);
    n[j] = at < prm.count ? (int)min((unsigned long long)kVec, prm.count - at) : 0;
    c[j] = load_codes(code + at, n[j], vec);
    e[j] = n[j] ? prm.scale[which][at / XP_STATE8_BLOCK] : 0;
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    O* to = out + first + j * (kDecodeCta / 2);
    if (n[j] == kVec && vec_out && pairs_ok(c[j], e[j])) {
      unsigned w[kVec / 2];
      if (which == 0)
        decode_pairs<true>(c[j], e[j], w);
      else
        decode_pairs<false>(c[j], e[j], w);
      if constexpr (sizeof(O) == 2) {
        *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        float2 f[kVec / 2];
        widen_pairs(w, f);
        reinterpret_cast<float4*>(to)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        reinterpret_cast<float4*>(to)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
      }
    } else if (n[j]) {
      float f[kVec];
      if (which == 0)
        decode_codes<true>(c[j], e[j], f);
      else
        decode_codes<false>(c[j], e[j], f);
      store_some(to, n[j], vec_out, f);
    }
  }
}

template <typename P, typename G, bool S8>
cudaError_t run_adamw(const StepParams& p, unsigned nunits, cudaStream_t st) {
  return launch_dependent(adamw_kernel<P, G, S8>, dim3(nunits), kStepThreads + kBooksThreads<S8>, 0, 1, st, p);
}

}  // namespace

cudaError_t launch_adamw(const StepParams& p, unsigned nunits, int param_dtype, int grad_dtype, int state_dtype,
                         cudaStream_t st) {
  typedef __nv_bfloat16 H;
  const bool s8 = state_dtype == XP_U8;
  if (param_dtype == XP_F32) {
    if (grad_dtype == XP_F32) return s8 ? run_adamw<float, float, true>(p, nunits, st) : run_adamw<float, float, false>(p, nunits, st);
    return s8 ? run_adamw<float, H, true>(p, nunits, st) : run_adamw<float, H, false>(p, nunits, st);
  }
  if (grad_dtype == XP_F32) return s8 ? run_adamw<H, float, true>(p, nunits, st) : run_adamw<H, float, false>(p, nunits, st);
  return s8 ? run_adamw<H, H, true>(p, nunits, st) : run_adamw<H, H, false>(p, nunits, st);
}

cudaError_t launch_grad_norm(const NormParams& p, int grad_dtype, cudaStream_t st) {
  const unsigned grid = p.nunits < (unsigned)kNormMaxCtas ? p.nunits : (unsigned)kNormMaxCtas;
  return launch_dependent(grad_dtype == XP_F32 ? grad_norm_kernel<float> : grad_norm_kernel<__nv_bfloat16>, dim3(grid), kNormThreads, 0, 1, st, p);
}

cudaError_t launch_set_grads(const SetGradsParams& p, cudaStream_t st) {
  return launch_dependent(set_grads_kernel, dim3(1), 256, 0, 1, st, p);
}

cudaError_t launch_set_step(GroupState* s, unsigned long long step, double p1, double p2, cudaStream_t st) {
  return launch_dependent(set_step_kernel, dim3(1), 1, 0, 1, st, s, step, p1, p2);
}

cudaError_t launch_decode(const DecodeParams& p, int out_dtype, cudaStream_t st) {
  const dim3 grid((unsigned)((p.count + kDecodeCta - 1) / kDecodeCta), 2);
  return launch_dependent(out_dtype == XP_F32 ? decode_kernel<float> : decode_kernel<__nv_bfloat16>, grid, kStepThreads, 0, 1, st, p);
}

}  // namespace xp
