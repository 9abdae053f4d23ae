// Passes over rows of logits that the distillation and the verification of
// drafted tokens share: a row's largest logit and its sum of exponentials in
// one pass, and the teacher's side of a distillation row.
#pragma once
#include <cfloat>

#include "spmv_device.cuh"
#include "spmv_types.cuh"

namespace spmv {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_fast(float x) {  // (2^-22 relative; 0 below 2^-126)
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Tokens of a row are passed in units of 8 from the row's first 16-byte
// boundary on, `head` single tokens before them and `tail` ones behind.
constexpr int kUnit = 8;

struct Units {
  int head, units, tail;
};

template <typename T>
__device__ __forceinline__ Units units_of(const T* row, int n) {
  const int to_line =
      (int)((16u - (unsigned)(reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) / (int)sizeof(T);
  Units u;
  u.head = min(to_line, n);
  u.units = (n - u.head) / kUnit;
  u.tail = n - u.head - u.units * kUnit;
  return u;
}

// The largest of a set of logits and sum(exp2((logit - largest) * c)) over
// it, joined as the set grows. Starting from the lowest finite number keeps
// the differences of minus infinities defined: they count as 0. (The
// difference is taken before the product with c: exact for near logits, and
// no overflow at the ends of fp32's range.)
struct MaxSum {
  float m, s;
  static __device__ __forceinline__ MaxSum none() { return {-FLT_MAX, 0.f}; }
  __device__ __forceinline__ void raise(float to, float c) {
    if (to > m) {
      s *= exp2_fast((m - to) * c);
      m = to;
    }
  }
  __device__ __forceinline__ void join(const MaxSum& o, float c) {
    raise(o.m, c);
    s += o.s * exp2_fast((o.m - m) * c);
  }
  __device__ __forceinline__ void add(const float (&v)[kUnit], float c) {
    float top = v[0];
#pragma unroll
    for (int k = 1; k < kUnit; ++k) top = fmaxf(top, v[k]);
    raise(top, c);
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int k = 0; k < kUnit; k += 2) {
      a += exp2_fast((v[k] - m) * c);
      b += exp2_fast((v[k + 1] - m) * c);
    }
    s += a + b;
  }
};

template <typename T>
__device__ __forceinline__ void widen(const Pack<T, kUnit>& r, float (&v)[kUnit]) {
#pragma unroll
  for (int k = 0; k < kUnit / 2; ++k) {
    const float2 p = pair_f32(r, k);
    v[2 * k] = p.x;
    v[2 * k + 1] = p.y;
  }
}

// f(first token of a unit, its 8 logits) over tokens [0, n) of a row by the
// THREADS threads of a CTA; places outside the row hold minus infinity (the
// head and the tail are units of their own). kAtOnce loads of a thread are
// under way together.
template <int THREADS, int AT_ONCE, typename T, typename F>
__device__ __forceinline__ void for_units(const T* row, int n, F&& f) {
  const Units u = units_of(row, n);
  const T* body = row + u.head;
  for (int k = threadIdx.x; k < u.units; k += AT_ONCE * THREADS) {
    Pack<T, kUnit> r[AT_ONCE];
#pragma unroll
    for (int h = 0; h < AT_ONCE; ++h)
      if (k + h * THREADS < u.units) r[h] = load_pack<T, kUnit>(body + (int64_t)(k + h * THREADS) * kUnit, true);
#pragma unroll
    for (int h = 0; h < AT_ONCE; ++h)
      if (k + h * THREADS < u.units) {
        float v[kUnit];
        widen(r[h], v);
        f(u.head + (k + h * THREADS) * kUnit, v);
      }
  }
  // the ends, by the last warp's threads (whose share is the smallest)
  const int me = THREADS - 1 - (int)threadIdx.x;
  const bool front = me == 0 && u.head > 0, back = me == 1 && u.tail > 0;
  if (front || back) {
    const int at = front ? 0 : u.head + u.units * kUnit, m = front ? u.head : u.tail;
    float v[kUnit];
#pragma unroll
    for (int k = 0; k < kUnit; ++k) v[k] = k < m ? to_f32(row[at + k]) : -INFINITY;
    f(at, v);
  }
}

// Join a MaxSum over the CTA; the result is the same in all threads. Ends
// with the shared memory free for reuse after the next barrier.
template <int THREADS>
__device__ __forceinline__ MaxSum join_cta(MaxSum x, float c, MaxSum* s_red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    MaxSum y;
    y.m = __shfl_xor_sync(0xffffffffu, x.m, o);
    y.s = __shfl_xor_sync(0xffffffffu, x.s, o);
    // (both sides compute the same: the larger first)
    const float m = fmaxf(x.m, y.m);
    x.s = x.s * exp2_fast((x.m - m) * c) + y.s * exp2_fast((y.m - m) * c);
    x.m = m;
  }
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = x;
  __syncthreads();
  MaxSum t = s_red[0];
#pragma unroll
  for (int w = 1; w < THREADS / 32; ++w) t.join(s_red[w], c);
  return t;
}

}  // namespace
}  // namespace spmv
