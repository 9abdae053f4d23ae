// Passes over rows of logits that the distillation and the verification of
// drafted tokens share: a row's largest logit and its sum of exponentials in
// one pass, and the teacher's side of a distillation row.
#pragma once
#include <cfloat>

#include "spmv_device.cuh"
#include "spmv_pairs.cuh"
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

// The larger of three, as one instruction (NaN is passed over, as fmaxf does).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The 8 logits of a unit, in pairs.
struct Unit {
  F2 p[kUnit / 2];
  __device__ __forceinline__ float largest() const {
    const float2 a = unpack2(p[0]), b = unpack2(p[1]), c = unpack2(p[2]), d = unpack2(p[3]);
    return fmaxf(max3(max3(a.x, a.y, b.x), b.y, c.x), max3(c.y, d.x, d.y));
  }
  // minus infinity where `marks` has a bit
  __device__ __forceinline__ void drop(uint32_t marks) {
#pragma unroll
    for (int k = 0; k < kUnit / 2; ++k) {
      const float2 v = unpack2(p[k]);
      p[k] = pack2(marks >> (2 * k) & 1 ? -INFINITY : v.x, marks >> (2 * k + 1) & 1 ? -INFINITY : v.y);
    }
  }
};

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
};

// The same for the units of a thread, the sum in two parts.
struct UnitSum {
  float m;
  F2 s;
  static __device__ __forceinline__ UnitSum none() { return {-FLT_MAX, 0}; }
  __device__ __forceinline__ void add(const Unit& u, float c) {
    const float top = u.largest();
    if (top > m) {
      s = mul2(s, both(exp2_fast((m - top) * c)));
      m = top;
    }
    const F2 nm = both(-m), cc = both(c);
#pragma unroll
    for (int k = 0; k < kUnit / 2; ++k) {
      const float2 a = unpack2(mul2(add2(u.p[k], nm), cc));
      s = add2(s, pack2(exp2_fast(a.x), exp2_fast(a.y)));
    }
  }
  __device__ __forceinline__ MaxSum sum() const {
    const float2 t = unpack2(s);
    return {m, t.x + t.y};
  }
};

template <typename T>
__device__ __forceinline__ Unit widen(const Pack<T, kUnit>& r) {
  Unit u;
#pragma unroll
  for (int k = 0; k < kUnit / 2; ++k) {
    const float2 p = pair_f32(r, k);
    u.p[k] = pack2(p.x, p.y);
  }
  return u;
}

// f(first token of a unit, its 8 logits) over tokens [0, n) of a row by the
// THREADS threads of a CTA; places outside the row hold minus infinity (the
// head and the tail are units of their own). AT_ONCE loads of a thread are
// under way together.
template <int THREADS, int AT_ONCE, typename T, typename F>
__device__ __forceinline__ void for_units(const T* row, int n, F&& f) {
  const Units u = units_of(row, n);
  const T* body = row + u.head;
  int k = threadIdx.x;
  for (; k + (AT_ONCE - 1) * THREADS < u.units; k += AT_ONCE * THREADS) {
    Pack<T, kUnit> r[AT_ONCE];
#pragma unroll
    for (int h = 0; h < AT_ONCE; ++h) r[h] = load_pack<T, kUnit>(body + (int64_t)(k + h * THREADS) * kUnit, true);
#pragma unroll
    for (int h = 0; h < AT_ONCE; ++h) {
      Unit v = widen(r[h]);
      f(u.head + (k + h * THREADS) * kUnit, v);
    }
  }
  {
    Pack<T, kUnit> r[AT_ONCE - 1];
#pragma unroll
    for (int h = 0; h < AT_ONCE - 1; ++h)
      if (k + h * THREADS < u.units) r[h] = load_pack<T, kUnit>(body + (int64_t)(k + h * THREADS) * kUnit, true);
#pragma unroll
    for (int h = 0; h < AT_ONCE - 1; ++h)
      if (k + h * THREADS < u.units) {
        Unit v = widen(r[h]);
        f(u.head + (k + h * THREADS) * kUnit, v);
      }
  }
  // the ends, by the last warp's threads (whose share is the smallest)
  const int me = THREADS - 1 - (int)threadIdx.x;
  const bool front = me == 0 && u.head > 0, back = me == 1 && u.tail > 0;
  if (front || back) {
    const int at = front ? 0 : u.head + u.units * kUnit, m = front ? u.head : u.tail;
    Unit v;
#pragma unroll
    for (int j = 0; j < kUnit / 2; ++j)
      v.p[j] = pack2(2 * j < m ? to_f32(row[at + 2 * j]) : -INFINITY, 2 * j + 1 < m ? to_f32(row[at + 2 * j + 1]) : -INFINITY);
    f(at, v);
  }
}

// Joined over LANES neighbouring lanes, the same in all of them.
template <int LANES>
__device__ __forceinline__ MaxSum join_lanes(MaxSum x, float c) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    const MaxSum y{__shfl_xor_sync(0xffffffffu, x.m, o), __shfl_xor_sync(0xffffffffu, x.s, o)};
    const float m = fmaxf(x.m, y.m);
    x.s = x.s * exp2_fast((x.m - m) * c) + y.s * exp2_fast((y.m - m) * c);
    x.m = m;
  }
  return x;
}

// Join a MaxSum over the CTA; the result is the same in all threads. Ends
// with the shared memory free for reuse after the next barrier.
template <int THREADS>
__device__ __forceinline__ MaxSum join_cta(MaxSum x, float c, MaxSum* s_red) {
  constexpr int kWarps = THREADS / 32;
  x = join_lanes<32>(x, c);
  if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = x;
  __syncthreads();
  return join_lanes<kWarps>(s_red[threadIdx.x % kWarps], c);
}

}  // namespace
}  // namespace spmv
