// Penalties, biases and grammar masks on logits (spmv_logits_process).
//
// Bound by reading the logits and writing them: 8 bytes per token of the
// vocabulary in fp32, against a few thousand list entries per request. Which
// tokens a request's lists hold, and how often, has to be known before its
// logits pass through: a table of one word per token in shared memory, for a
// share of the vocabulary per CTA. Every CTA reads the whole lists for its
// share, from L2: an eighth to a sixth more traffic there at a few thousand
// entries, and none in memory. (Sharing the reading among a cluster, with
// counts in distributed shared memory, measured slower: 95 against 289 us
// where this takes XX on 256 requests of 128000 tokens.) Requests whose
// parameters change nothing skip the tables.
#include <climits>
#include <type_traits>

#include "spmv_device.cuh"
#include "spmv_types.cuh"

namespace spmv {
namespace {

constexpr int kLogitThreads = 512, kLogitWarps = kLogitThreads / 32;
constexpr int kShare = 16384;      // tokens of a CTA's table, at most (64 KB)
constexpr int kLeastShare = 1024;  // and at least
constexpr int kListed = 512;       // biases of a CTA's share kept in shared memory
// table word: output tokens in the low 30 bits, and
constexpr uint32_t kSeen = 0x80000000u, kBiased = 0x40000000u, kCount = 0x3fffffffu;

constexpr int kWave = 2 * 152;  // CTAs that the device's SMs hold at a time, two each

struct LogitArgs {
  spmv_logits l;
  int shares;  // per request
  int share;   // tokens of each (a multiple of 32)
};

struct Penalty {
  float rep, freq, pres;
};

__device__ __forceinline__ float penalised(float l, uint32_t w, const Penalty& c) {
  if (w & (kSeen | kCount)) l = l > 0.f ? l / c.rep : l * c.rep;
  if (w & kCount) l = l - c.freq * (float)(w & kCount) - c.pres;
  return l;
}

// A request's lists and parameters. Lists that would change nothing are empty.
struct Request {
  Penalty c;
  int64_t p0, p1, o0, o1, b0, b1;
  int mask_row;  // -1: none
  __device__ __forceinline__ void load(const spmv_logits& p, int64_t i) {
    c.rep = p.repetition ? p.repetition[i] : 1.f;
    c.freq = p.frequency ? p.frequency[i] : 0.f;
    c.pres = p.presence ? p.presence[i] : 0.f;
    p0 = p1 = o0 = o1 = b0 = b1 = 0;
    if (p.prompt_tokens) p0 = p.prompt_offsets[i], p1 = p.prompt_offsets[i + 1];
    if (p.output_tokens) o0 = p.output_offsets[i], o1 = p.output_offsets[i + 1];
    if (p.bias_tokens) b0 = p.bias_offsets[i], b1 = p.bias_offsets[i + 1];
    mask_row = p.mask ? (p.mask_rows ? p.mask_rows[i] : (int)i) : -1;
    if (mask_row >= p.n_masks) mask_row = -1;
    if (c.rep == 1.f) {
      p1 = p0;
      if (c.freq == 0.f && c.pres == 0.f) o1 = o0;
    }
  }
};

// CTAs take (request, share of the vocabulary) pairs in turn. While one passes
// through, the next one's parameters and first list entries come into
// registers and its logits into L2. A table is cleared as it is read, so it is
// empty again for the next pair.
template <typename T, typename OT, int VEC>
__global__ void __launch_bounds__(kLogitThreads, 2) logits_rows(LogitArgs a) {
  extern __shared__ __align__(16) uint32_t s_word[];  // a.share words
  __shared__ int s_token[kListed];
  __shared__ float s_value[kListed];
  __shared__ int s_warp[kLogitWarps];
  constexpr int kBatch = VEC == 1 ? 8 : 4;  // vectors under way per thread
  constexpr int kFirst = 4;                 // prompt entries loaded ahead per thread
  const spmv_logits& p = a.l;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, me = threadIdx.x;
  const int64_t jobs = (int64_t)p.n_requests * a.shares;
  const auto ask_logits = [&](int64_t i, int v0) {
    const int n = min(a.share, p.vocab - v0);
    const char* at =
        reinterpret_cast<const char*>(static_cast<const T*>(p.logits) + i * p.stride + v0);
    for (int64_t k = 128ll * me; k < n * (int64_t)sizeof(T); k += 128 * kLogitThreads)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(at + k));
  };
  struct First {
    int prompt[kFirst], output, bias;
    float value;
  };
  const auto load_first = [&](const Request& q, First& f) {
#pragma unroll
    for (int h = 0; h < kFirst; ++h) {
      const int64_t k = q.p0 + me + h * kLogitThreads;
      f.prompt[h] = k < q.p1 ? p.prompt_tokens[k] : -1;
    }
    f.output = q.o0 + me < q.o1 ? p.output_tokens[q.o0 + me] : -1;
    const bool on = q.b0 + me < q.b1;
    f.bias = on ? p.bias_tokens[q.b0 + me] : -1;
    f.value = on ? p.bias_values[q.b0 + me] : 0.f;
  };
  int64_t i = blockIdx.x / (unsigned)a.shares;
  int v0 = (int)(blockIdx.x % (unsigned)a.shares) * a.share;
  const int64_t step_i = gridDim.x / (unsigned)a.shares;
  const int step_v = (int)(gridDim.x % (unsigned)a.shares) * a.share, wrap = a.shares * a.share;
  ask_logits(i, v0);
  Request next;
  First first_next;
  next.load(p, i);
  for (int k = 4 * me; k < a.share; k += 4 * kLogitThreads)
    *reinterpret_cast<uint4*>(s_word + k) = make_uint4(0, 0, 0, 0);
  load_first(next, first_next);
  __syncthreads();

  for (int64_t id = blockIdx.x; id < jobs; id += gridDim.x) {
    const int n = min(a.share, p.vocab - v0);
    const T* in = static_cast<const T*>(p.logits) + i * p.stride + v0;
    OT* out = static_cast<OT*>(p.out) + i * p.out_stride + v0;
    const Request q = next;
    const First f = first_next;
    int64_t next_i = i + step_i;
    int next_v = v0 + step_v;
    if (next_v >= wrap) next_v -= wrap, ++next_i;
    const bool more = id + gridDim.x < jobs;
    if (more) next.load(p, next_i);
    const uint32_t* mask = q.mask_row >= 0 ? p.mask + q.mask_row * p.mask_stride + v0 / 32 : nullptr;
    const bool counted = q.p1 > q.p0 || q.o1 > q.o0;
    if (counted) {
      const auto seen = [&](int v) {
        if (v >= v0 && v < v0 + n) atomicOr(s_word + (v - v0), kSeen);
      };
      const auto told = [&](int v) {
        if (v >= v0 && v < v0 + n) atomicAdd(s_word + (v - v0), 1u);
      };
      constexpr int kAtOnce = 4;
      for (int64_t k = q.p0 + me + kFirst * kLogitThreads; k < q.p1; k += kAtOnce * kLogitThreads) {
        int v[kAtOnce];
#pragma unroll
        for (int h = 0; h < kAtOnce; ++h)
          v[h] = k + h * kLogitThreads < q.p1 ? p.prompt_tokens[k + h * kLogitThreads] : -1;
#pragma unroll
        for (int h = 0; h < kAtOnce; ++h) seen(v[h]);
      }
      for (int64_t k = q.o0 + me + kLogitThreads; k < q.o1; k += kAtOnce * kLogitThreads) {
        int v[kAtOnce];
#pragma unroll
        for (int h = 0; h < kAtOnce; ++h)
          v[h] = k + h * kLogitThreads < q.o1 ? p.output_tokens[k + h * kLogitThreads] : -1;
#pragma unroll
        for (int h = 0; h < kAtOnce; ++h) told(v[h]);
      }
#pragma unroll
      for (int h = 0; h < kFirst; ++h) seen(f.prompt[h]);
      told(f.output);
    }
    if (more) {
      ask_logits(next_i, next_v);
      load_first(next, first_next);
    }
    // biases of this CTA's tokens, compacted in list order
    int listed = 0;
    for (int64_t k = q.b0; k < q.b1; k += kLogitThreads) {
      int v = f.bias;
      float value = f.value;
      if (k > q.b0) {
        const bool on = k + me < q.b1;
        v = on ? p.bias_tokens[k + me] : -1;
        value = on ? p.bias_values[k + me] : 0.f;
      }
      const bool mine = v >= v0 && v < v0 + n;
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
      if (mine && before < kListed) {
        s_token[before] = v;
        s_value[before] = value;
      }
      listed += total;
      __syncthreads();
    }
    if (counted) __syncthreads();
    const auto allowed = [&](int k) { return !mask || (mask[k / 32] >> (k % 32) & 1u); };
    if (listed > 0) {
      // A token with biases is finished by the thread of its first entry and
      // marked, so that the pass below leaves it alone.
      const auto finish = [&](int v, float sum) {
        const int k = v - v0;
        const uint32_t w = atomicOr(s_word + k, kBiased);
        out[k] = from_f32<OT>(allowed(k) ? penalised(to_f32(in[k]), w, q.c) + sum : -INFINITY);
      };
      if (listed <= kListed) {
        if ((int)threadIdx.x < listed) {
          const int v = s_token[threadIdx.x];
          float sum = 0.f;
          bool first = true;
          for (int k = 0; k < listed; ++k) {
            if (s_token[k] != v) continue;
            first = first && k >= (int)threadIdx.x;
            sum += s_value[k];
          }
          if (first) finish(v, sum);
        }
      } else {  // more than the compacted list holds: from the list itself
        for (int64_t at = q.b0 + threadIdx.x; at < q.b1; at += kLogitThreads) {
          const int v = p.bias_tokens[at];
          if (v < v0 || v >= v0 + n) continue;
          float sum = 0.f;
          bool first = true;
          for (int64_t k = q.b0; k < q.b1 && first; ++k) {
            if (p.bias_tokens[k] != v) continue;
            first = k >= at;
            sum += p.bias_values[k];
          }
          if (first) finish(v, sum);
        }
      }
      __syncthreads();
    }
    const bool table = counted || listed > 0;
    for (int base = VEC * threadIdx.x; base < n; base += kBatch * VEC * kLogitThreads) {
      Pack<T, VEC> v[kBatch];
      uint32_t bits[kBatch];  // of the tokens from k on (VEC of them, within one word)
#pragma unroll
      for (int h = 0; h < kBatch; ++h) {
        const int k = base + h * VEC * kLogitThreads;
        if (k < n) v[h] = load_pack<T, VEC>(in + k, true);
      }
#pragma unroll
      for (int h = 0; h < kBatch; ++h) {
        const int k = base + h * VEC * kLogitThreads;
        bits[h] = mask && k < n ? __ldg(mask + k / 32) >> (k % 32) : 0xffffffffu;
      }
#pragma unroll
      for (int h = 0; h < kBatch; ++h) {
        const int k = base + h * VEC * kLogitThreads;
        if (k >= n) break;
        Pack<uint32_t, VEC> w = {};
        if (table) {
          w = load_pack<uint32_t, VEC>(s_word + k);
          store_pack<uint32_t, VEC>(s_word + k, Pack<uint32_t, VEC>{});
        }
        Pack<OT, VEC> r;
        uint32_t any = 0;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          float l = to_f32(v[h].v[e]);
          if (w.v[e]) l = penalised(l, w.v[e], q.c);  // (few tokens of a vocabulary)
          r.v[e] = from_f32<OT>(bits[h] >> e & 1 ? l : -INFINITY);
          any |= w.v[e];
        }
        if (!(any & kBiased)) {
          store_pack<OT, VEC>(out + k, r);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (!(w.v[e] & kBiased)) out[k + e] = r.v[e];
        }
      }
    }
    __syncthreads();  // the table is empty, the list of biases done with
    i = next_i;
    v0 = next_v;
  }
}

template <typename T, typename OT>
spmv_status launch_logits(const spmv_logits& p, cudaStream_t st) {
  LogitArgs a{};
  a.l = p;
  // As large a share as a table holds, every list being read once for each
  // share; smaller ones where the requests would not give every SM two CTAs.
  const int64_t tokens = (int64_t)p.vocab * p.n_requests / kWave;
  const int64_t per = tokens < kLeastShare ? kLeastShare : tokens > kShare ? kShare : tokens;
  a.shares = (int)((p.vocab + per - 1) / per);
  a.share = (int)(((int64_t)p.vocab + a.shares - 1) / a.shares + 31) / 32 * 32;
  a.shares = (int)(((int64_t)p.vocab + a.share - 1) / a.share);
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
  const int64_t jobs = (int64_t)p.n_requests * a.shares;
  void* args[] = {&a};
  return cudaLaunchKernel(fn, dim3((unsigned)(jobs < kWave ? jobs : kWave)), dim3(kLogitThreads),
                          args, smem, st) == cudaSuccess
             ? SPMV_OK
             : SPMV_ERR_CUDA;
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
