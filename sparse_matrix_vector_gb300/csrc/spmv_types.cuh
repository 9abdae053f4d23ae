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
