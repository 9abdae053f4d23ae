// Penalties, biases and grammar masks on logits (spmv_logits_process).
//
// Bound by reading the logits and writing them: 8 bytes per token of the
// vocabulary in fp32, against a few thousand list entries per request. Which
// tokens a request's lists hold, and how often, has to be known before its
// logits pass through: a table of one word per token, which a cluster of CTAs
// holds in its shared memory, each CTA the words of its share of the
// vocabulary. Every CTA reads a share of the lists and counts into the owners'
// tables (integer atomics in distributed shared memory: the order does not
// matter), while its share of the logits is on its way into L2. Requests
// whose parameters change nothing skip the tables.
#include <cooperative_groups.h>

#include <climits>
#include <type_traits>

#include "spmv_device.cuh"
#include "spmv_types.cuh"

namespace spmv {
namespace {

namespace cg = cooperative_groups;

constexpr int kLogitThreads = 512, kLogitWarps = kLogitThreads / 32;
constexpr int kShare = 16384;      // tokens of a CTA's table, at most (64 KB: three CTAs per SM)
constexpr int kLogitCluster = 8;   // CTAs that share a request's range, at most
constexpr int kListed = 512;       // biases of a CTA's share kept in shared memory
// table word: output tokens in the low 30 bits, and
constexpr uint32_t kSeen = 0x80000000u, kBiased = 0x40000000u, kCount = 0x3fffffffu;

struct LogitArgs {
  spmv_logits l;
  int ranges;  // clusters per request, each with its range of the vocabulary
  int share;   // tokens per CTA (a multiple of 32)
};

struct Penalty {
  float rep, freq, pres;
};

__device__ __forceinline__ float penalised(float l, uint32_t w, const Penalty& c) {
  if (w & (kSeen | kCount)) l = l > 0.f ? l / c.rep : l * c.rep;
  if (w & kCount) l = l - c.freq * (float)(w & kCount) - c.pres;
  return l;
}

// Sum of a token's biases in list order: over the CTA's compacted list, or
// over the request's whole list where that did not fit.
__device__ __noinline__ float bias_of(const spmv_logits& p, int token, int64_t b0, int64_t b1,
                                         const int* s_token, const float* s_value, int listed) {
  float sum = 0.f;
  if (listed <= kListed) {
    for (int k = 0; k < listed; ++k)
      if (s_token[k] == token) sum += s_value[k];
  } else {
    for (int64_t k = b0; k < b1; ++k)
      if (p.bias_tokens[k] == token) sum += p.bias_values[k];
  }
  return sum;
}

template <typename T, typename OT, int VEC>
__global__ void __launch_bounds__(kLogitThreads, VEC == 8 ? 2 : 3) logits_rows(LogitArgs a) {
  extern __shared__ __align__(16) uint32_t s_word[];  // a.share words
  __shared__ int s_token[kListed];
  __shared__ float s_value[kListed];
  __shared__ int s_warp[kLogitWarps];
  const spmv_logits& p = a.l;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), cta = cluster.block_rank();
  const int id = blockIdx.x / ctas, i = id / a.ranges;
  // tokens [r0, r1) of the cluster, [v0, v1) of this CTA
  const int r0 = (id % a.ranges) * (a.share * ctas);
  const int r1 = (int)min((int64_t)p.vocab, (int64_t)r0 + a.share * ctas);
  const int v0 = min(r0 + cta * a.share, r1), v1 = min(v0 + a.share, r1), n = v1 - v0;
  const T* in = static_cast<const T*>(p.logits) + i * p.stride + v0;
  OT* out = static_cast<OT*>(p.out) + i * p.out_stride + v0;
  for (int64_t k = 128ll * threadIdx.x; k < n * (int64_t)sizeof(T); k += 128 * kLogitThreads)
    asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const char*>(in) + k));

  const Penalty c{p.repetition ? p.repetition[i] : 1.f, p.frequency ? p.frequency[i] : 0.f,
                  p.presence ? p.presence[i] : 0.f};
  const bool has_prompt = p.prompt_tokens && c.rep != 1.f;
  const bool has_output = p.output_tokens && (c.rep != 1.f || c.freq != 0.f || c.pres != 0.f);
  const int64_t p0 = has_prompt ? p.prompt_offsets[i] : 0, p1 = has_prompt ? p.prompt_offsets[i + 1] : 0;
  const int64_t o0 = has_output ? p.output_offsets[i] : 0, o1 = has_output ? p.output_offsets[i + 1] : 0;
  const int64_t b0 = p.bias_tokens ? p.bias_offsets[i] : 0, b1 = p.bias_tokens ? p.bias_offsets[i + 1] : 0;
  const int row = p.mask ? (p.mask_rows ? p.mask_rows[i] : i) : -1;
  const uint32_t* mask =
      row >= 0 && row < p.n_masks ? p.mask + row * p.mask_stride + v0 / 32 : nullptr;
  const bool counted = p1 > p0 || o1 > o0, biased = b1 > b0;  // (the same in the whole cluster)
  int listed = 0;
  if (counted || biased) {
    for (int k = 4 * threadIdx.x; k < n; k += 4 * kLogitThreads)
      *reinterpret_cast<uint4*>(s_word + k) = make_uint4(0, 0, 0, 0);
    if (counted) {
      cluster.sync();
      const int me = cta * kLogitThreads + threadIdx.x, all = ctas * kLogitThreads;
      const auto word = [&](int v) {  // null outside the cluster's range
        const unsigned at = (unsigned)(v - r0);
        return v >= r0 && v < r1
                   ? cluster.map_shared_rank(s_word, at / (unsigned)a.share) + at % (unsigned)a.share
                   : nullptr;
      };
#pragma unroll 4
      for (int64_t k = p0 + me; k < p1; k += all)
        if (uint32_t* w = word(p.prompt_tokens[k])) atomicOr(w, kSeen);
#pragma unroll 4
      for (int64_t k = o0 + me; k < o1; k += all)
        if (uint32_t* w = word(p.output_tokens[k])) atomicAdd(w, 1u);
      cluster.sync();
    } else {
      __syncthreads();
    }
    // biases of this CTA's tokens, in list order
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t k = b0; k < b1; k += kLogitThreads) {
      const int64_t at = k + threadIdx.x;
      const int v = at < b1 ? p.bias_tokens[at] : -1;
      const float value = at < b1 ? p.bias_values[at] : 0.f;
      const bool mine = v >= v0 && v < v1;
      const uint32_t m = __ballot_sync(0xffffffffu, mine);
      if (lane == 0) s_warp[warp] = __popc(m);
      __syncthreads();
      int before = listed, total = 0;
#pragma unroll
      for (int w = 0; w < kLogitWarps; ++w) {
        before += w < warp ? s_warp[w] : 0;
        total += s_warp[w];
      }
      before += __popc(m & ((1u << lane) - 1));
      if (mine) {
        atomicOr(s_word + (v - v0), kBiased);
        if (before < kListed) {
          s_token[before] = v;
          s_value[before] = value;
        }
      }
      listed += total;
      __syncthreads();
    }
  }
  const bool table = counted || listed > 0;
  const auto finished = [&](float l, uint32_t w, int k) {
    l = penalised(l, w, c);
    if (w & kBiased) l += bias_of(p, v0 + k, b0, b1, s_token, s_value, listed);
    return l;
  };
#pragma unroll 2
  for (int k = VEC * threadIdx.x; k < n; k += VEC * kLogitThreads) {
    const Pack<T, VEC> v = load_pack<T, VEC>(in + k, true);
    // bits of the tokens from k on (VEC of them, within one word)
    const uint32_t bits = mask ? __ldg(mask + k / 32) >> (k % 32) : 0xffffffffu;
    Pack<uint32_t, VEC> w = {};
    if (table) w = load_pack<uint32_t, VEC>(s_word + k);
    Pack<OT, VEC> r;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float l = to_f32(v.v[e]);
      if (w.v[e]) l = finished(l, w.v[e], k + e);  // (few tokens of a vocabulary)
      r.v[e] = from_f32<OT>(bits >> e & 1 ? l : -INFINITY);
    }
    store_pack<OT, VEC>(out + k, r);
  }
}

template <typename T, typename OT>
spmv_status launch_logits(const spmv_logits& p, cudaStream_t st) {
  LogitArgs a{};
  a.l = p;
  // shares of at least 2048 tokens, clusters of up to 8 of them
  int ctas = 1;
  while (ctas < kLogitCluster && (int64_t)ctas * 2048 < p.vocab) ctas *= 2;
  const int64_t per = (p.vocab + (int64_t)ctas - 1) / ctas;
  a.share = (int)((per < kShare ? per : kShare) + 31) / 32 * 32;
  a.ranges = (int)((p.vocab + (int64_t)a.share * ctas - 1) / ((int64_t)a.share * ctas));
  const int64_t grid = (int64_t)p.n_requests * a.ranges * ctas;
  if (grid > INT_MAX) return SPMV_ERR_TOO_LARGE;
  constexpr int kVec = 16 / (int)sizeof(T);
  const bool vec = p.vocab % kVec == 0 &&
                   rows_aligned(p.logits, p.n_requests, p.stride, sizeof(T), kVec) &&
                   rows_aligned(p.out, p.n_requests, p.out_stride, sizeof(OT), kVec);
  const void* fn = vec ? reinterpret_cast<const void*>(&logits_rows<T, OT, kVec>)
                       : reinterpret_cast<const void*>(&logits_rows<T, OT, 1>);
  const size_t smem = (size_t)a.share * 4;
  if (smem > 40 * 1024 &&  // 48 KB less the static part need no opt-in
      cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
          cudaSuccess)
    return SPMV_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kLogitThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {&a};
  return cudaLaunchKernelExC(&cfg, fn, args) == cudaSuccess ? SPMV_OK : SPMV_ERR_CUDA;
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
  const bool wide = p.out_dtype == SPMV_F32;
  if (p.dtype == SPMV_F32) return launch_logits<float, float>(p, st);
  if (p.dtype == SPMV_F16)
    return wide ? launch_logits<__half, float>(p, st) : launch_logits<__half, __half>(p, st);
  return wide ? launch_logits<__nv_bfloat16, float>(p, st)
              : launch_logits<__nv_bfloat16, __nv_bfloat16>(p, st);
}
