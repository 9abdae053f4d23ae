// Low-rank adapters of many requests beside a shared projection
// (spmv_adapters_run): y_t = base_t + scale_s * B_s (A_s x_t), s the slot of
// token t.
#include <climits>

#include "spmv_device.cuh"
#include "spmv_types.cuh"

namespace spmv {
namespace {

struct AdapterArgs {
  int n_tokens, n_in, n_out, n_slots, rank;
  const void* x;
  int64_t xs;
  const void *a, *b;
  const int32_t *ids, *ranks;
  const float* scales;
  const void* base;
  int64_t bs;
  void* y;
  int64_t ys;
  float* h;  // n_tokens x rank
};

// Slot of token t (-1: none) and its rank.
__device__ __forceinline__ int slot_of(const AdapterArgs& p, int t, int* rank) {
  const int s = p.ids[t];
  if (s < 0 || s >= p.n_slots) return -1;
  *rank = p.ranks ? min(max(p.ranks[s], 0), p.rank) : p.rank;
  return s;
}

// h = A_s x_t: a warp per (row of A, token).
template <typename T>
__global__ void __launch_bounds__(kThreads) adapters_shrink(AdapterArgs p) {
  const int t = blockIdx.x, j = blockIdx.y * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  int rank = 0;
  const int s = slot_of(p, t, &rank);
  if (s < 0 || j >= rank) return;
  const T* x = static_cast<const T*>(p.x) + t * p.xs;
  const T* a = static_cast<const T*>(p.a) + ((int64_t)s * p.rank + j) * p.n_in;
  float v = 0.f;
  for (int k = lane; k < p.n_in; k += 32) v += to_f32(a[k]) * to_f32(x[k]);
  v = warp_sum(v);
  if (lane == 0) p.h[(int64_t)t * p.rank + j] = v;
}

// y = base + scale * B_s h: a thread per (column, token).
template <typename T, typename YT>
__global__ void __launch_bounds__(kThreads) adapters_expand(AdapterArgs p) {
  __shared__ float s_h[SPMV_ADAPTER_MAX_RANK];
  const int t = blockIdx.x, o = blockIdx.y * kThreads + threadIdx.x;
  int rank = 0;
  const int s = slot_of(p, t, &rank);
  if (s >= 0)
    for (int j = threadIdx.x; j < rank; j += kThreads) s_h[j] = p.h[(int64_t)t * p.rank + j];
  __syncthreads();
  if (o >= p.n_out) return;
  float v = 0.f;
  if (s >= 0) {
    const T* b = static_cast<const T*>(p.b) + ((int64_t)s * p.n_out + o) * p.rank;
    for (int j = 0; j < rank; ++j) v += to_f32(b[j]) * s_h[j];
    if (p.scales) v *= p.scales[s];
  }
  const float base = p.base ? to_f32(static_cast<const YT*>(p.base)[t * p.bs + o]) : 0.f;
  static_cast<YT*>(p.y)[t * p.ys + o] = from_f32<YT>(s >= 0 ? base + v : base);
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" int64_t spmv_adapters_workspace(int32_t n_tokens, int32_t n_slots, int32_t rank) {
  if (n_tokens < 0 || n_slots < 0 || rank < 0 || rank > SPMV_ADAPTER_MAX_RANK ||
      n_slots > SPMV_ADAPTER_MAX_SLOTS)
    return 0;
  return n_slots > 0 ? (int64_t)n_tokens * rank * 4 : 0;
}

extern "C" spmv_status spmv_adapters_run(int32_t n_tokens, int32_t n_in, int32_t n_out,
                                         int32_t n_slots, int32_t rank, spmv_dtype dtype,
                                         const void* x, int64_t x_stride, const void* a,
                                         const void* b, const int32_t* slot_ids,
                                         const int32_t* ranks, const float* scales,
                                         const void* base, int64_t base_stride, void* y,
                                         spmv_dtype y_dtype, int64_t y_stride, void* workspace,
                                         int64_t workspace_bytes, void* stream) {
  if (n_tokens < 0 || n_in < 0 || n_out < 0 || n_slots < 0 || rank < 0 || !op_dtype(dtype) ||
      !op_dtype(y_dtype))
    return SPMV_ERR_INVALID_ARG;
  if (dtype == SPMV_F32 || (y_dtype != SPMV_F32 && y_dtype != dtype)) return SPMV_ERR_UNSUPPORTED;
  if (rank > SPMV_ADAPTER_MAX_RANK || n_slots > SPMV_ADAPTER_MAX_SLOTS) return SPMV_ERR_TOO_LARGE;
  const int64_t ysz = op_dtype_size(y_dtype);
  const bool weights = n_slots > 0 && rank > 0;
  if (!matrix_ok(x, n_tokens, n_in, x_stride, 2, false) ||
      (base && !matrix_ok(base, n_tokens, n_out, base_stride, ysz, false)) ||
      !matrix_ok(y, n_tokens, n_out, y_stride, ysz, true) ||
      (weights && ((n_in > 0 && !a) || (n_out > 0 && !b))) || !aligned_to(a, 2) ||
      !aligned_to(b, 2) || (n_tokens > 0 && !slot_ids) || !aligned_to(slot_ids, 4) ||
      !aligned_to(ranks, 4) || !aligned_to(scales, 4) || !aligned_to(workspace, 16))
    return SPMV_ERR_INVALID_ARG;
  const int64_t need = spmv_adapters_workspace(n_tokens, n_slots, rank);
  if (need > 0 && (!workspace || workspace_bytes < need)) return SPMV_ERR_INVALID_ARG;
  if (n_tokens == 0 || n_out == 0) return SPMV_OK;
  const bool in_place = base == y && (base_stride == y_stride || n_tokens == 1);
  if ((!in_place && spans_overlap(base, n_tokens, n_out, base_stride, ysz, y, n_tokens, n_out,
                                  y_stride, ysz)) ||
      spans_overlap(x, n_tokens, n_in, x_stride, 2, y, n_tokens, n_out, y_stride, ysz))
    return SPMV_ERR_INVALID_ARG;
  AdapterArgs p{n_tokens, n_in,   n_out, n_slots,     rank, x,        x_stride, a,
                b,        slot_ids, ranks, scales,    base, base_stride, y,     y_stride,
                static_cast<float*>(workspace)};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const dim3 shrink(n_tokens, (rank + kWarps - 1) / kWarps);
  const dim3 expand(n_tokens, (n_out + kThreads - 1) / kThreads);
  if (weights) {
    if (dtype == SPMV_F16)
      adapters_shrink<__half><<<shrink, kThreads, 0, st>>>(p);
    else
      adapters_shrink<__nv_bfloat16><<<shrink, kThreads, 0, st>>>(p);
  }
  if (dtype == SPMV_F16 && y_dtype == SPMV_F32)
    adapters_expand<__half, float><<<expand, kThreads, 0, st>>>(p);
  else if (dtype == SPMV_F16)
    adapters_expand<__half, __half><<<expand, kThreads, 0, st>>>(p);
  else if (y_dtype == SPMV_F32)
    adapters_expand<__nv_bfloat16, float><<<expand, kThreads, 0, st>>>(p);
  else
    adapters_expand<__nv_bfloat16, __nv_bfloat16><<<expand, kThreads, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SPMV_OK : SPMV_ERR_CUDA;
}
