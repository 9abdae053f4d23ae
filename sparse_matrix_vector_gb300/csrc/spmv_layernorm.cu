// Layer norm of rows and its gradient (spmv_layernorm,
// spmv_layernorm_backward).
#include <climits>

#include "spmv_device.cuh"
#include "spmv_types.cuh"

namespace spmv {
namespace {

// Sum over the CTA, in every thread. Fixed order.
__device__ __forceinline__ float cta_sum_all(float v, float* s_red) {
  const float t = cta_sum(v, s_red);
  __syncthreads();
  if (threadIdx.x == 0) s_red[0] = t;
  __syncthreads();
  const float r = s_red[0];
  __syncthreads();
  return r;
}

// One row per CTA step; three passes over the row (mean, variance, output).
template <typename XT, typename YT>
__global__ void __launch_bounds__(kThreads)
layernorm_rows(int64_t n_rows, int n_cols, const XT* x, int64_t xs, const void* w, const void* b,
               int pt, float eps, YT* y, int64_t ys, float* mean_out, float* rstd_out) {
  __shared__ float s_red[kWarps];
  for (int64_t r = blockIdx.x; r < n_rows; r += gridDim.x) {
    const XT* xr = x + r * xs;
    YT* yr = y + r * ys;
    float s = 0.f;
    for (int j = threadIdx.x; j < n_cols; j += kThreads) s += to_f32(xr[j]);
    const float mean = cta_sum_all(s, s_red) / (float)n_cols;
    float q = 0.f;
    for (int j = threadIdx.x; j < n_cols; j += kThreads) {
      const float c = to_f32(xr[j]) - mean;
      q += c * c;
    }
    const float rstd = rsqrtf(cta_sum_all(q, s_red) / (float)n_cols + eps);
    for (int j = threadIdx.x; j < n_cols; j += kThreads) {
      const float g = w ? load_as_f32(w, pt, j) : 1.f, o = b ? load_as_f32(b, pt, j) : 0.f;
      yr[j] = from_f32<YT>((to_f32(xr[j]) - mean) * rstd * g + o);
    }
    if (threadIdx.x == 0) {
      if (mean_out) mean_out[r] = mean;
      if (rstd_out) rstd_out[r] = rstd;
    }
  }
}

// dx, one row per CTA step.
template <typename XT, typename YT>
__global__ void __launch_bounds__(kThreads)
layernorm_dx_rows(int64_t n_rows, int n_cols, const YT* dy, int64_t dys, const XT* x, int64_t xs,
                  const void* w, int pt, const float* mean, const float* rstd, XT* dx,
                  int64_t dxs) {
  __shared__ float s_red[kWarps];
  for (int64_t r = blockIdx.x; r < n_rows; r += gridDim.x) {
    const float m = mean[r], rs = rstd[r];
    float sg = 0.f, sgx = 0.f;
    for (int j = threadIdx.x; j < n_cols; j += kThreads) {
      const float g = to_f32(dy[r * dys + j]) * (w ? load_as_f32(w, pt, j) : 1.f);
      sg += g;
      sgx += g * ((to_f32(x[r * xs + j]) - m) * rs);
    }
    sg = cta_sum_all(sg, s_red) / (float)n_cols;
    sgx = cta_sum_all(sgx, s_red) / (float)n_cols;
    for (int j = threadIdx.x; j < n_cols; j += kThreads) {
      const float g = to_f32(dy[r * dys + j]) * (w ? load_as_f32(w, pt, j) : 1.f);
      const float xh = (to_f32(x[r * xs + j]) - m) * rs;
      dx[r * dxs + j] = from_f32<XT>(rs * (g - sg - xh * sgx));
    }
  }
}

// dweight and dbias of kThreads columns: partial sums of a block of rows,
// then (layernorm_params_sum) the blocks in order.
constexpr int kParamBlocks = 64;

template <typename XT, typename YT>
__global__ void __launch_bounds__(kThreads)
layernorm_params_part(int64_t n_rows, int n_cols, const YT* dy, int64_t dys, const XT* x,
                      int64_t xs, const float* mean, const float* rstd, float* part) {
  const int j = blockIdx.x * kThreads + threadIdx.x;
  if (j >= n_cols) return;
  const int64_t per = (n_rows + kParamBlocks - 1) / kParamBlocks;
  const int64_t lo = blockIdx.y * per, hi = lo + per < n_rows ? lo + per : n_rows;
  float dw = 0.f, db = 0.f;
  for (int64_t r = lo; r < hi; ++r) {
    const float d = to_f32(dy[r * dys + j]);
    dw += d * ((to_f32(x[r * xs + j]) - mean[r]) * rstd[r]);
    db += d;
  }
  part[(int64_t)blockIdx.y * 2 * n_cols + j] = dw;
  part[((int64_t)blockIdx.y * 2 + 1) * n_cols + j] = db;
}

__global__ void __launch_bounds__(kThreads)
layernorm_params_sum(int n_cols, const float* part, void* dw_out, void* db_out, int pt) {
  const int j = blockIdx.x * kThreads + threadIdx.x;
  if (j >= n_cols) return;
  float dw = 0.f, db = 0.f;
  for (int k = 0; k < kParamBlocks; ++k) {
    dw += part[(int64_t)k * 2 * n_cols + j];
    db += part[((int64_t)k * 2 + 1) * n_cols + j];
  }
  if (dw_out) store_from_f32(dw_out, pt, j, dw);
  if (db_out) store_from_f32(db_out, pt, j, db);
}

constexpr int kMaxCols = INT32_MAX - 4096;
constexpr int kRowGrid = 152 * 8;

template <typename F>
spmv_status by_types(spmv_dtype x, spmv_dtype y, F&& f) {
  if (x == SPMV_F32 && y == SPMV_F32) return f((float*)nullptr, (float*)nullptr);
  if (x == SPMV_F32 && y == SPMV_F16) return f((float*)nullptr, (__half*)nullptr);
  if (x == SPMV_F32 && y == SPMV_BF16) return f((float*)nullptr, (__nv_bfloat16*)nullptr);
  if (x == SPMV_F16 && y == SPMV_F16) return f((__half*)nullptr, (__half*)nullptr);
  if (x == SPMV_BF16 && y == SPMV_BF16)
    return f((__nv_bfloat16*)nullptr, (__nv_bfloat16*)nullptr);
  return SPMV_ERR_UNSUPPORTED;
}

int64_t backward_workspace(int64_t n_rows, int n_cols, bool want_params) {
  return want_params && n_rows > 0 ? (int64_t)kParamBlocks * 2 * n_cols * 4 : 0;
}

spmv_status launched() { return cudaGetLastError() == cudaSuccess ? SPMV_OK : SPMV_ERR_CUDA; }

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" spmv_status spmv_layernorm(int64_t n_rows, int32_t n_cols, const void* x,
                                      spmv_dtype x_dtype, int64_t x_stride, const void* weight,
                                      const void* bias, spmv_dtype param_dtype, float eps, void* y,
                                      spmv_dtype y_dtype, int64_t y_stride, float* mean_out,
                                      float* rstd_out, void* stream) {
  if (n_rows < 0 || n_cols < 1 || !op_dtype(x_dtype) || !op_dtype(y_dtype) ||
      !op_dtype(param_dtype) || !(eps >= 0.f) || !std::isfinite(eps))
    return SPMV_ERR_INVALID_ARG;
  if (x_dtype != SPMV_F32 && y_dtype != x_dtype) return SPMV_ERR_UNSUPPORTED;
  if (n_cols > kMaxCols) return SPMV_ERR_TOO_LARGE;
  const int64_t xs = op_dtype_size(x_dtype), ysz = op_dtype_size(y_dtype),
                ps = op_dtype_size(param_dtype);
  if (!matrix_ok(x, n_rows, n_cols, x_stride, xs, false) ||
      !matrix_ok(y, n_rows, n_cols, y_stride, ysz, true) || !aligned_to(weight, ps) ||
      !aligned_to(bias, ps) || !aligned_to(mean_out, 4) || !aligned_to(rstd_out, 4))
    return SPMV_ERR_INVALID_ARG;
  if (n_rows == 0) return SPMV_OK;
  const bool in_place = x == y && x_dtype == y_dtype && (x_stride == y_stride || n_rows == 1);
  if (!in_place &&
      spans_overlap(x, n_rows, n_cols, x_stride, xs, y, n_rows, n_cols, y_stride, ysz))
    return SPMV_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int grid = (int)(n_rows < kRowGrid ? n_rows : kRowGrid);
  return by_types(x_dtype, y_dtype, [&](auto* xt, auto* yt) {
    using XT = std::remove_pointer_t<decltype(xt)>;
    using YT = std::remove_pointer_t<decltype(yt)>;
    layernorm_rows<XT, YT><<<grid, kThreads, 0, st>>>(
        n_rows, n_cols, static_cast<const XT*>(x), x_stride, weight, bias, param_dtype, eps,
        static_cast<YT*>(y), y_stride, mean_out, rstd_out);
    return launched();
  });
}

extern "C" int64_t spmv_layernorm_backward_workspace(int64_t n_rows, int32_t n_cols,
                                                     int32_t want_params) {
  if (n_rows < 0 || n_cols < 1 || n_cols > kMaxCols) return 0;
  return backward_workspace(n_rows, n_cols, want_params != 0);
}

extern "C" spmv_status spmv_layernorm_backward(
    int64_t n_rows, int32_t n_cols, const void* dy, spmv_dtype dy_dtype, int64_t dy_stride,
    const void* x, spmv_dtype x_dtype, int64_t x_stride, const void* weight,
    spmv_dtype param_dtype, const float* mean, const float* rstd, void* dx, int64_t dx_stride,
    void* dweight, void* dbias, void* workspace, int64_t workspace_bytes, void* stream) {
  if (n_rows < 0 || n_cols < 1 || !op_dtype(x_dtype) || !op_dtype(dy_dtype) ||
      !op_dtype(param_dtype))
    return SPMV_ERR_INVALID_ARG;
  if (x_dtype != SPMV_F32 && dy_dtype != x_dtype) return SPMV_ERR_UNSUPPORTED;
  if (n_cols > kMaxCols) return SPMV_ERR_TOO_LARGE;
  const int64_t xs = op_dtype_size(x_dtype), dys = op_dtype_size(dy_dtype),
                ps = op_dtype_size(param_dtype);
  const bool params = dweight || dbias;
  if (!matrix_ok(x, n_rows, n_cols, x_stride, xs, false) ||
      !matrix_ok(dy, n_rows, n_cols, dy_stride, dys, false) ||
      (dx && !matrix_ok(dx, n_rows, n_cols, dx_stride, xs, true)) ||
      (n_rows > 0 && (!mean || !rstd)) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) ||
      !aligned_to(weight, ps) || !aligned_to(dweight, ps) || !aligned_to(dbias, ps) ||
      !aligned_to(workspace, 16))
    return SPMV_ERR_INVALID_ARG;
  const int64_t need = backward_workspace(n_rows, n_cols, params);
  if (need > 0 && (!workspace || workspace_bytes < need)) return SPMV_ERR_INVALID_ARG;
  const bool in_place = dx == dy && x_dtype == dy_dtype && (dx_stride == dy_stride || n_rows <= 1);
  if (dx && ((!in_place && spans_overlap(dx, n_rows, n_cols, dx_stride, xs, dy, n_rows, n_cols,
                                         dy_stride, dys)) ||
             spans_overlap(dx, n_rows, n_cols, dx_stride, xs, x, n_rows, n_cols, x_stride, xs)))
    return SPMV_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n_rows == 0) {
    if ((dweight && cudaMemsetAsync(dweight, 0, (size_t)(n_cols * ps), st) != cudaSuccess) ||
        (dbias && cudaMemsetAsync(dbias, 0, (size_t)(n_cols * ps), st) != cudaSuccess))
      return SPMV_ERR_CUDA;
    return SPMV_OK;
  }
  const int grid = (int)(n_rows < kRowGrid ? n_rows : kRowGrid);
  return by_types(x_dtype, dy_dtype, [&](auto* xt, auto* yt) {
    using XT = std::remove_pointer_t<decltype(xt)>;
    using YT = std::remove_pointer_t<decltype(yt)>;
    const int col_blocks = (n_cols + kThreads - 1) / kThreads;
    if (params) {
      float* part = static_cast<float*>(workspace);
      layernorm_params_part<XT, YT><<<dim3(col_blocks, kParamBlocks), kThreads, 0, st>>>(
          n_rows, n_cols, static_cast<const YT*>(dy), dy_stride, static_cast<const XT*>(x),
          x_stride, mean, rstd, part);
      layernorm_params_sum<<<col_blocks, kThreads, 0, st>>>(n_cols, part, dweight, dbias,
                                                            param_dtype);
    }
    if (dx)
      layernorm_dx_rows<XT, YT><<<grid, kThreads, 0, st>>>(
          n_rows, n_cols, static_cast<const YT*>(dy), dy_stride, static_cast<const XT*>(x),
          x_stride, weight, param_dtype, mean, rstd, static_cast<XT*>(dx), dx_stride);
    return launched();
  });
}
