// Element types of the operators around a pruned layer (fp32, fp16, bf16):
// conversions, 16-byte vectors, and the argument checks that their entry
// points share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <map>
#include <mutex>
#include <utility>

#include "spmv_device.cuh"
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

// This thread's asynchronous copies of 4, 8 or 16 bytes into shared memory,
// in groups; each thread reads back only what it copied itself, so waiting
// for its own groups is all the synchronisation there is.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src),
                 "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// Ask L2 for the whole 16-byte granules of [p, p + bytes), by one thread: one
// request to the copy engine. (The same by prefetches of single lines takes
// the load/store units a cycle or more per line, which the loads behind them
// wait for.)
__device__ __forceinline__ void prefetch_bulk(const void* p, int64_t bytes) {
  const uintptr_t lo = (reinterpret_cast<uintptr_t>(p) + 15) & ~uintptr_t(15);
  const uintptr_t hi = (reinterpret_cast<uintptr_t>(p) + (uintptr_t)bytes) & ~uintptr_t(15);
  if (bytes > 0 && hi > lo)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(lo), "r"((uint32_t)(hi - lo))
                 : "memory");
}

// ------------------------------------------------- a thread's columns of a row
// A group of `group` threads shares a row of n columns, thread `me` holding
// NV vectors of VEC (even) columns. ALIGNED: rows start on vector boundaries
// and n is a multiple of VEC; vector i is VEC neighbouring columns at
// (i * group + me) * VEC, moved as a whole. Otherwise element k of vector i
// is column (i * VEC + k) * group + me, moved element by element, so that a
// warp's accesses are still contiguous.
template <int VEC, bool ALIGNED>
struct Cols {
  int me, group, n;
  __device__ __forceinline__ int col(int i, int k) const {
    return ALIGNED ? (i * group + me) * VEC + k : (i * VEC + k) * group + me;
  }
  // whether vector i (ALIGNED) is inside the row
  __device__ __forceinline__ bool has(int i) const { return !ALIGNED || col(i, 0) < n; }
  __device__ __forceinline__ bool has(int i, int k) const { return ALIGNED || col(i, k) < n; }
  // Loads of all vectors, under way together: places past the end hold the
  // row's last vector (ALIGNED) or zeros.
  template <typename T, int NV>
  __device__ __forceinline__ void load(const T* row, Pack<T, VEC> (&r)[NV], bool stream) const {
    if constexpr (ALIGNED) {
#pragma unroll
      for (int i = 0; i < NV; ++i) r[i] = load_pack<T, VEC>(row + min(col(i, 0), n - VEC), stream);
    } else {
      const T* at = row + me;
#pragma unroll
      for (int j = 0; j < NV * VEC; ++j) {
        T v = from_f32<T>(0.f);
        if (me + j * group < n) v = load_pack<T, 1>(at, stream).v[0];
        r[j / VEC].v[j % VEC] = v;
        at += group;
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, int i, const Pack<T, VEC>& r) const {
    if constexpr (ALIGNED) {
      store_pack<T, VEC>(row + col(i, 0), r);
    } else {
      T* at = row + col(i, 0);
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        if (col(i, k) < n) *at = r.v[k];
        at += group;
      }
    }
  }
  // The same columns of a vector of runtime type (a layer's parameter), in
  // fp32; `fill` for a null pointer.
  template <typename T, int NV>
  __device__ __forceinline__ void load_as(const void* p, float2 (&v)[NV][VEC / 2]) const {
    Pack<T, VEC> r[NV];
    load<T, NV>(static_cast<const T*>(p), r, false);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int k = 0; k < VEC / 2; ++k)
        v[i][k] = make_float2(to_f32(r[i].v[2 * k]), to_f32(r[i].v[2 * k + 1]));
  }
  template <int NV>
  __device__ __forceinline__ void load_param(const void* p, int dtype, float fill,
                                             float2 (&v)[NV][VEC / 2]) const {
    if (!p) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VEC / 2; ++k) v[i][k] = make_float2(fill, fill);
    } else if (dtype == SPMV_F32) {
      load_as<float, NV>(p, v);
    } else if (dtype == SPMV_F16) {
      load_as<__half, NV>(p, v);
    } else {
      load_as<__nv_bfloat16, NV>(p, v);
    }
  }
  // Ask L2 for a row (its loads come one row later).
  template <typename T>
  __device__ __forceinline__ void prefetch(const T* row) const {
    if (me == 0) prefetch_bulk(row, (int64_t)n * (int)sizeof(T));
  }
};

// Elements 2k and 2k + 1 of a vector, in fp32.
template <typename T, int N>
__device__ __forceinline__ float2 pair_f32(const Pack<T, N>& r, int k) {
  return make_float2(to_f32(r.v[2 * k]), to_f32(r.v[2 * k + 1]));
}
template <int N>
__device__ __forceinline__ float2 pair_f32(const Pack<__nv_bfloat16, N>& r, int k) {
  // bf16 is the upper half of an fp32
  const uint32_t w = reinterpret_cast<const uint32_t*>(&r)[k];
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <int N>
__device__ __forceinline__ float2 pair_f32(const Pack<__half, N>& r, int k) {
  return __half22float2(reinterpret_cast<const __half2*>(&r)[k]);
}
template <int N>
__device__ __forceinline__ void set_pair(Pack<float, N>& r, int k, float2 v) {
  r.v[2 * k] = v.x;
  r.v[2 * k + 1] = v.y;
}
template <int N>
__device__ __forceinline__ void set_pair(Pack<__half, N>& r, int k, float2 v) {
  reinterpret_cast<__half2*>(&r)[k] = __float22half2_rn(v);
}
template <int N>
__device__ __forceinline__ void set_pair(Pack<__nv_bfloat16, N>& r, int k, float2 v) {
  reinterpret_cast<__nv_bfloat162*>(&r)[k] = __float22bfloat162_rn(v);
}

}  // namespace

// The status of a runtime call or a launch, from its own result: the error
// that the runtime keeps for the thread may be an earlier call's. One of this
// call is reported here, and not left there for a later one.
inline spmv_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return SPMV_OK;
  cudaGetLastError();
  return SPMV_ERR_CUDA;
}
// (of launch helpers that give 0 or -1)
inline spmv_status status_of_launch(int e) {
  return status_of(e == 0 ? cudaSuccess : cudaErrorLaunchFailure);
}

// Launch fn(p).
template <typename Args>
spmv_status launch(void (*fn)(Args), dim3 grid, int threads, size_t smem, cudaStream_t st,
                   const Args& p) {
  void* args[] = {const_cast<Args*>(&p)};
  return status_of(cudaLaunchKernel(reinterpret_cast<const void*>(fn), grid, dim3((unsigned)threads),
                                    args, smem, st));
}

// Leave for a kernel to be launched with `bytes` of dynamic shared memory.
// The limit belongs to the function and counts for all host threads, and a
// launch beyond it is refused: so it is set once per kernel and device, to the
// most that the device has beside the kernel's static part, and never lowered.
inline bool allow_smem(const void* fn, size_t bytes) {
  if (bytes <= 16 * 1024) return true;  // (48 KB less any static part need no leave)
  static std::mutex mu;
  static std::map<std::pair<const void*, int>, size_t> most;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  std::lock_guard<std::mutex> lock(mu);
  const auto known = most.find({fn, dev});
  if (known != most.end()) return bytes <= known->second;
  int optin = 0;
  cudaFuncAttributes attr;
  if (cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) !=
          cudaSuccess ||
      cudaFuncGetAttributes(&attr, fn) != cudaSuccess ||
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           optin - (int)attr.sharedSizeBytes) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  const size_t room = (size_t)optin - attr.sharedSizeBytes;
  most[{fn, dev}] = room;
  return bytes <= room;
}

// Clusters of `cluster` CTAs that the current device holds at a time: what
// fits its SMs by registers and shared memory, less what a cluster's being
// confined to one group of SMs leaves over (36 rather than 38 clusters of 8
// at two CTAs per SM). Asked once per kernel and launch shape. 0 on error.
inline int resident_clusters(const void* fn, int cluster, int block, size_t smem) {
  struct Known {
    const void* fn;
    int dev, cluster;
    size_t smem;
    int n;
  };
  static std::mutex mu;
  static Known known[128];
  static int count = 0;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < count; ++i)
    if (known[i].fn == fn && known[i].dev == dev && known[i].cluster == cluster &&
        known[i].smem == smem)
      return known[i].n;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)cluster);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (!allow_smem(fn, smem) ||
      cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    return 0;
  }
  if (count < 128) known[count++] = Known{fn, dev, cluster, smem, n};
  return n;
}

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

// Rows of a matrix that vectors of `vec` elements can be loaded from: every
// row starts on a whole vector (of at most 16 bytes).
inline bool rows_aligned(const void* p, int64_t rows, int64_t stride, int64_t size, int vec) {
  const int64_t bytes = size * vec > 16 ? 16 : size * vec;
  return aligned_to(p, bytes) && (rows <= 1 || (stride * size) % bytes == 0);
}

// Whether two matrices may share bytes. Where their spans meet, rows of one
// distance may still be column ranges of one matrix, side by side, or rows of
// it in turn: then they share bytes only if some do modulo that distance.
inline bool spans_overlap(const void* p, int64_t p_rows, int64_t p_cols, int64_t p_stride,
                          int64_t p_size, const void* q, int64_t q_rows, int64_t q_cols,
                          int64_t q_stride, int64_t q_size) {
  if (!p || !q || p_rows == 0 || q_rows == 0 || p_cols == 0 || q_cols == 0) return false;
  const uintptr_t p0 = (uintptr_t)p, q0 = (uintptr_t)q;
  const uintptr_t p1 = p0 + (uintptr_t)(((p_rows - 1) * p_stride + p_cols) * p_size);
  const uintptr_t q1 = q0 + (uintptr_t)(((q_rows - 1) * q_stride + q_cols) * q_size);
  if (p0 >= q1 || q0 >= p1) return false;
  const uintptr_t p_row = (uintptr_t)(p_cols * p_size), q_row = (uintptr_t)(q_cols * q_size);
  const uintptr_t p_step = (uintptr_t)(p_stride * p_size), q_step = (uintptr_t)(q_stride * q_size);
  const uintptr_t step = p_rows > 1 ? p_step : q_step;
  if ((p_rows == 1 && q_rows == 1) || (p_rows > 1 && q_rows > 1 && p_step != q_step) ||
      p_row > step || q_row > step)
    return true;
  const uintptr_t d = q0 >= p0 ? (q0 - p0) % step : (step - (p0 - q0) % step) % step;
  return d < p_row || d + q_row > step;
}

}  // namespace spmv
