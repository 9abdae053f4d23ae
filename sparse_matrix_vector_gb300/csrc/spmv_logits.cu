// Penalties, biases and grammar masks on logits (spmv_logits_process).
#include <climits>

#include "spmv_device.cuh"
#include "spmv_types.cuh"

namespace spmv {
namespace {

constexpr int kSlice = 4096;  // tokens of the vocabulary per CTA

// A CTA per (request, slice of the vocabulary): it counts the request's
// tokens that fall into its slice in shared memory (output tokens in the low
// 31 bits, seen in the top bit), applies the penalties, then adds up the
// biases of the slice and applies the mask.
template <typename T, typename OT>
__global__ void __launch_bounds__(kThreads) logits_slices(spmv_logits p, int slices) {
  __shared__ uint32_t s_count[kSlice];
  __shared__ float s_bias[kSlice];
  const int i = blockIdx.x / slices, lo = (blockIdx.x % slices) * kSlice;
  const int n = min(kSlice, p.vocab - lo);
  for (int k = threadIdx.x; k < n; k += kThreads) {
    s_count[k] = 0;
    s_bias[k] = 0.f;
  }
  __syncthreads();
  if (p.prompt_tokens)
    for (int64_t k = p.prompt_offsets[i] + threadIdx.x; k < p.prompt_offsets[i + 1]; k += kThreads) {
      const unsigned v = (unsigned)(p.prompt_tokens[k] - lo);
      if (p.prompt_tokens[k] >= lo && v < (unsigned)n) atomicOr(&s_count[v], 0x80000000u);
    }
  if (p.output_tokens)
    for (int64_t k = p.output_offsets[i] + threadIdx.x; k < p.output_offsets[i + 1]; k += kThreads) {
      const unsigned v = (unsigned)(p.output_tokens[k] - lo);
      if (p.output_tokens[k] >= lo && v < (unsigned)n) atomicAdd(&s_count[v], 1u);
    }
  // one thread keeps the list's order
  if (p.bias_tokens && threadIdx.x == 0)
    for (int64_t k = p.bias_offsets[i]; k < p.bias_offsets[i + 1]; ++k) {
      const int v = p.bias_tokens[k];
      if (v >= lo && v - lo < n) s_bias[v - lo] += p.bias_values[k];
    }
  __syncthreads();
  const float rep = p.repetition ? p.repetition[i] : 1.f;
  const float freq = p.frequency ? p.frequency[i] : 0.f, pres = p.presence ? p.presence[i] : 0.f;
  const int row = p.mask ? (p.mask_rows ? p.mask_rows[i] : i) : -1;
  const bool masked = row >= 0 && row < p.n_masks;
  for (int k = threadIdx.x; k < n; k += kThreads) {
    float l = to_f32(static_cast<const T*>(p.logits)[i * p.stride + lo + k]);
    const uint32_t c = s_count[k];
    if (c) l = l > 0.f ? l / rep : l * rep;
    if (c & 0x7fffffffu) l = l - freq * (float)(c & 0x7fffffffu) - pres;
    l += s_bias[k];
    if (masked && !((p.mask[row * p.mask_stride + ((lo + k) >> 5)] >> ((lo + k) & 31)) & 1u))
      l = -INFINITY;
    static_cast<OT*>(p.out)[i * p.out_stride + lo + k] = from_f32<OT>(l);
  }
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" spmv_status spmv_logits_process(const spmv_logits* args, void* stream) {
  if (!args) return SPMV_ERR_INVALID_ARG;
  const spmv_logits& p = *args;
  if (p.n_requests < 0 || p.vocab < 0 || p.n_masks < 0 || !op_dtype(p.dtype) ||
      !op_dtype(p.out_dtype))
    return SPMV_ERR_INVALID_ARG;
  if (p.out_dtype != SPMV_F32 && p.out_dtype != p.dtype) return SPMV_ERR_UNSUPPORTED;
  const int64_t xs = op_dtype_size(p.dtype), os = op_dtype_size(p.out_dtype);
  if (!matrix_ok(p.logits, p.n_requests, p.vocab, p.stride, xs, false) ||
      !matrix_ok(p.out, p.n_requests, p.vocab, p.out_stride, os, true) ||
      (p.mask && !matrix_ok(p.mask, p.n_masks, (p.vocab + 31ll) / 32, p.mask_stride, 4, false)) ||
      (p.prompt_tokens && !p.prompt_offsets) || (p.output_tokens && !p.output_offsets) ||
      (p.bias_tokens && (!p.bias_offsets || !p.bias_values)))
    return SPMV_ERR_INVALID_ARG;
  const void* words[] = {p.prompt_tokens, p.output_tokens, p.repetition, p.frequency,
                         p.presence,      p.bias_tokens,   p.bias_values, p.mask_rows};
  for (const void* w : words)
    if (!aligned_to(w, 4)) return SPMV_ERR_INVALID_ARG;
  if (!aligned_to(p.prompt_offsets, 8) || !aligned_to(p.output_offsets, 8) ||
      !aligned_to(p.bias_offsets, 8))
    return SPMV_ERR_INVALID_ARG;
  if (p.n_requests == 0 || p.vocab == 0) return SPMV_OK;
  const bool in_place = p.logits == p.out && p.dtype == p.out_dtype &&
                        (p.stride == p.out_stride || p.n_requests == 1);
  if (!in_place && spans_overlap(p.logits, p.n_requests, p.vocab, p.stride, xs, p.out,
                                 p.n_requests, p.vocab, p.out_stride, os))
    return SPMV_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int slices = (p.vocab - 1) / kSlice + 1;
  if ((int64_t)slices * p.n_requests > INT_MAX) return SPMV_ERR_TOO_LARGE;
  const int grid = slices * p.n_requests;
  const auto launch = [&](auto* t, auto* o) {
    using T = std::remove_pointer_t<decltype(t)>;
    using OT = std::remove_pointer_t<decltype(o)>;
    logits_slices<T, OT><<<grid, kThreads, 0, st>>>(p, slices);
  };
  const bool wide = p.out_dtype == SPMV_F32;
  if (p.dtype == SPMV_F32)
    launch((float*)nullptr, (float*)nullptr);
  else if (p.dtype == SPMV_F16)
    wide ? launch((__half*)nullptr, (float*)nullptr) : launch((__half*)nullptr, (__half*)nullptr);
  else
    wide ? launch((__nv_bfloat16*)nullptr, (float*)nullptr)
         : launch((__nv_bfloat16*)nullptr, (__nv_bfloat16*)nullptr);
  return cudaGetLastError() == cudaSuccess ? SPMV_OK : SPMV_ERR_CUDA;
}
