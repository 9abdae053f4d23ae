// Element types of the operators around a pruned layer (fp32, fp16, bf16):
// conversions, 16-byte vectors, and the argument checks that their entry
// points share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "spmv_internal.h"

namespace spmv {
namespace {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Element i of an array of runtime type (weights, biases and their
// gradients: few elements, whose type is not worth a kernel of its own).
__device__ __forceinline__ float load_as_f32(const void* p, int dtype, int64_t i) {
  if (dtype == SPMV_F32) return static_cast<const float*>(p)[i];
  if (dtype == SPMV_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void store_from_f32(void* p, int dtype, int64_t i, float v) {
  if (dtype == SPMV_F32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == SPMV_F16)
    static_cast<__half*>(p)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

// N elements as one or two vector loads (N * sizeof(T) of 2, 4, 8, 16 or 32
// bytes, aligned to it, at most 16), widened to fp32. `stream`: data that is
// read once and should leave the caches first.
template <int BYTES>
struct Bits;
template <>
struct Bits<2> { using type = unsigned short; };
template <>
struct Bits<4> { using type = unsigned; };
template <>
struct Bits<8> { using type = uint2; };
template <>
struct Bits<16> { using type = uint4; };

template <typename T, int N>
struct alignas(N * sizeof(T) > 16 ? 16 : N * sizeof(T)) Pack {
  T v[N];
};

template <typename T, int N>
__device__ __forceinline__ Pack<T, N> load_pack(const T* p, bool stream = false) {
  constexpr int kBytes = N * (int)sizeof(T), kPart = kBytes > 16 ? 16 : kBytes;
  using B = typename Bits<kPart>::type;
  Pack<T, N> r;
#pragma unroll
  for (int i = 0; i < kBytes / kPart; ++i) {
    const B* q = reinterpret_cast<const B*>(p) + i;
    reinterpret_cast<B*>(&r)[i] = stream ? __ldcs(q) : *q;
  }
  return r;
}

template <typename T, int N>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, N>& r) {
  constexpr int kBytes = N * (int)sizeof(T), kPart = kBytes > 16 ? 16 : kBytes;
  using B = typename Bits<kPart>::type;
#pragma unroll
  for (int i = 0; i < kBytes / kPart; ++i)
    reinterpret_cast<B*>(p)[i] = reinterpret_cast<const B*>(&r)[i];
}

// VEC elements at column c of a row of n: a vector past the end repeats the
// last one (an unconditional load, so that loads of several vectors go out
// together); a single element past the end is zero.
template <typename T, int VEC>
__device__ __forceinline__ Pack<T, VEC> load_vec(const T* row, int c, int n, bool stream) {
  if constexpr (VEC == 1) {
    Pack<T, VEC> r;
    r.v[0] = from_f32<T>(0.f);
    if (c < n) r = load_pack<T, VEC>(row + c, stream);
    return r;
  } else {
    return load_pack<T, VEC>(row + min(c, n - VEC), stream);
  }
}

// A thread's columns of a vector of runtime type, as fp32: vectors of VEC
// columns at first + i * step, i < NV (as load_vec past the end); `fill` for a null pointer. The type is tested once, so that
// all of the loads are under way together.
template <typename T, int NV, int VEC>
__device__ __forceinline__ void load_cols_as(const T* p, int first, int step, int n,
                                             float (&v)[NV][VEC]) {
  Pack<T, VEC> r[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) r[i] = load_vec<T, VEC>(p, first + i * step, n, false);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < VEC; ++k) v[i][k] = to_f32(r[i].v[k]);
}

template <int NV, int VEC>
__device__ __forceinline__ void load_cols(const void* p, int dtype, int first, int step, int n,
                                          float fill, float (&v)[NV][VEC]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[i][k] = fill;
  } else if (dtype == SPMV_F32) {
    load_cols_as<float, NV, VEC>(static_cast<const float*>(p), first, step, n, v);
  } else if (dtype == SPMV_F16) {
    load_cols_as<__half, NV, VEC>(static_cast<const __half*>(p), first, step, n, v);
  } else {
    load_cols_as<__nv_bfloat16, NV, VEC>(static_cast<const __nv_bfloat16*>(p), first, step, n, v);
  }
}

}  // namespace

inline bool op_dtype(int t) { return t == SPMV_F32 || t == SPMV_F16 || t == SPMV_BF16; }
inline int64_t op_dtype_size(int t) { return t == SPMV_F32 ? 4 : 2; }
inline bool aligned_to(const void* p, int64_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes) == 0;
}

// A matrix argument: rows of `cols` elements of `size` bytes, `stride`
// elements apart. False if the pointer is null or misaligned, or the stride
// is negative, makes output rows overlap, or passes 63-bit byte offsets.
inline bool matrix_ok(const void* p, int64_t rows, int64_t cols, int64_t stride, int64_t size,
                      bool output) {
  if (rows == 0 || cols == 0) return true;
  if (!p || !aligned_to(p, size) || stride < 0) return false;
  if (output && rows > 1 && stride < cols) return false;
  return rows <= 1 || stride == 0 || rows <= (INT64_MAX / 16) / stride;
}

// Whether the bytes of two matrices' spans overlap.
inline bool spans_overlap(const void* p, int64_t p_rows, int64_t p_cols, int64_t p_stride,
                          int64_t p_size, const void* q, int64_t q_rows, int64_t q_cols,
                          int64_t q_stride, int64_t q_size) {
  if (!p || !q || p_rows == 0 || q_rows == 0 || p_cols == 0 || q_cols == 0) return false;
  const uintptr_t p0 = (uintptr_t)p, q0 = (uintptr_t)q;
  const uintptr_t p1 = p0 + (uintptr_t)(((p_rows - 1) * p_stride + p_cols) * p_size);
  const uintptr_t q1 = q0 + (uintptr_t)(((q_rows - 1) * q_stride + q_cols) * q_size);
  return p0 < q1 && q0 < p1;
}

}  // namespace spmv
