// Penalties, biases and grammar masks on logits (spmv_logits_process).
//
// Bound by reading the logits and writing them: 8 bytes per token of the
// vocabulary in fp32, against a few thousand list entries per request. Which
// tokens a request's lists hold, and how often, takes a table in shared
// memory, for a share of the vocabulary per CTA; every CTA reads the whole
// lists for its share, from L2. The few tokens that are listed are finished
// one by one before the share passes through and are put in place after it, so
// that the pass itself is a copy with a mask. Requests whose parameters change
// nothing skip the tables.
//
// Measured: 256 x 128000 fp32 with histories of up to 8192 tokens and 300
// biases 75 us, 0.53 of the 6.79 TB/s of a plain copy; with empty lists 50
// (0.77). A share's lists are a chain of waits (entries, atomics on the table,
// the listed logits) of some 6 us in each of four rounds of shares, which the
// SM's other two CTAs hide in part. 32000 of one request: 8.0 us, of which a
// launch is 4. Shares with more than kListed biases take longer (finish_many).
#include <climits>
#include <type_traits>

#include "spmv_device.cuh"
#include "spmv_types.cuh"

namespace spmv {
namespace {

constexpr int kLogitThreads = 384, kLogitWarps = kLogitThreads / 32;
constexpr int kLogitPerSm = 3;  // CTAs: one passes logits through while others are at their lists
// A token's 16 bits of the table: count among the output tokens (exact below
// kHeavy, which it passes by no more than a CTA's threads), and marks.
constexpr uint32_t kSeen = 0x8000u, kBiased = 0x4000u, kCount = 0x3fffu, kHeavy = 0x2000u;
constexpr int kShare = 20480;      // tokens of a CTA's share, at most (a table of 40 KB)
constexpr int kLeastShare = 1024;  // and at least
constexpr int kMet = 2048;         // listed tokens of a share kept as a list, with their results
constexpr int kListed = 384;       // biases kept in shared memory at a time
constexpr int kMany = 1 << 20;     // added to the count of met tokens of a share with more of them

constexpr int kWave = kLogitPerSm * 152;  // CTAs that the device's SMs hold at a time

struct LogitArgs {
  spmv_logits l;
  int shares;  // per request
  int share;   // tokens of each (a multiple of 32)
};

struct Penalty {
  float rep, freq, pres;
};

__device__ __forceinline__ float penalised(float l, bool seen, int64_t count, const Penalty& c) {
  if (seen || count > 0) l = l > 0.f ? l / c.rep : l * c.rep;
  if (count > 0) l = l - c.freq * (float)count - c.pres;
  return l;
}

// A request's lists and parameters. Lists that would change nothing are empty.
struct Request {
  Penalty c;
  int64_t p0, p1, o0, o1, b0, b1;
  int mask_row;  // -1: none
  // (settle() waits for what load() has only asked for)
  __device__ __forceinline__ void load(const spmv_logits& p, int64_t i) {
    c.rep = p.repetition ? p.repetition[i] : 1.f;
    c.freq = p.frequency ? p.frequency[i] : 0.f;
    c.pres = p.presence ? p.presence[i] : 0.f;
    p0 = p1 = o0 = o1 = b0 = b1 = 0;
    if (p.prompt_tokens) p0 = p.prompt_offsets[i], p1 = p.prompt_offsets[i + 1];
    if (p.output_tokens) o0 = p.output_offsets[i], o1 = p.output_offsets[i + 1];
    if (p.bias_tokens) b0 = p.bias_offsets[i], b1 = p.bias_offsets[i + 1];
    mask_row = p.mask ? (p.mask_rows ? p.mask_rows[i] : (int)i) : -1;
  }
  __device__ __forceinline__ void settle(const spmv_logits& p) {
    if (mask_row >= p.n_masks) mask_row = -1;
    if (c.rep == 1.f) {
      p1 = p0;
      if (c.freq == 0.f && c.pres == 0.f) o1 = o0;
    }
  }
};

// Put the lanes' tokens k that are `met` for the first time on the list: one
// atomic per warp (one per token queued up on the counter's address).
__device__ __forceinline__ void list_met(bool met, int k, int* s_n, uint16_t* s_met) {
  const uint32_t m = __ballot_sync(0xffffffffu, met);
  if (m == 0) return;
  const int lane = threadIdx.x & 31;
  int at = 0;
  if (lane == 0) at = atomicAdd(s_n, __popc(m));
  at = __shfl_sync(0xffffffffu, at, 0);
  at += __popc(m & ((1u << lane) - 1));
  if (met && at < kMet) s_met[at] = (uint16_t)k;
}

// f(entry - v0) for every entry of list[lo, hi) inside [v0, v0 + n), by the
// whole CTA, 16 bytes of the list at a time where it allows that; f says
// whether it meets the token for the first time. Most entries belong to other
// shares: a warp first queues its own ones, so that f runs with all lanes at
// work.
constexpr int kQueue = 256;

template <typename F>
__device__ __forceinline__ void for_entries(const int32_t* list, int64_t lo, int64_t hi, int v0,
                                            int n, uint16_t* queue, int* s_n,
                                            uint16_t* s_met, F&& f) {
  if (lo >= hi) return;
  const int me = threadIdx.x, lane = me & 31;
  const uint32_t below = (1u << lane) - 1;
  int queued = 0;  // (the same in all lanes)
  const auto flush = [&] {
    __syncwarp();
    for (int e = 0; e < queued; e += 32) {
      const bool on = e + lane < queued;
      const int k = on ? queue[e + lane] : 0;
      list_met(on && f(k), k, s_n, s_met);
    }
    __syncwarp();
    queued = 0;
  };
  const auto offer = [&](int v) {
    const unsigned at = (unsigned)v - (unsigned)v0;
    const uint32_t m = __ballot_sync(0xffffffffu, at < (unsigned)n);
    if (at < (unsigned)n) queue[queued + __popc(m & below)] = (uint16_t)at;
    queued += __popc(m);
  };
  const int to_line = (int)((0u - (unsigned)(reinterpret_cast<uintptr_t>(list + lo) >> 2)) & 3u);
  const int head = (int)min((int64_t)to_line, hi - lo);
  const int64_t vecs = (hi - lo - head) / 4;
  const int4* body = reinterpret_cast<const int4*>(list + lo + head);
  int edge = -1;  // an entry before or after the vectors
  const int tail = (int)(hi - lo - head - 4 * vecs);
  if (me < head) edge = list[lo + me];
  if (me >= 4 && me - 4 < tail) edge = list[hi - tail + me - 4];
  constexpr int kAtOnce = 4;
  for (int64_t k = me - lane; k < vecs; k += kAtOnce * kLogitThreads) {  // (whole warps)
    int4 v[kAtOnce];
#pragma unroll
    for (int h = 0; h < kAtOnce; ++h)
      v[h] = k + lane + h * kLogitThreads < vecs ? __ldg(body + k + lane + h * kLogitThreads)
                                                 : make_int4(-1, -1, -1, -1);
#pragma unroll
    for (int h = 0; h < kAtOnce; ++h) {
      if (queued > kQueue - 128) flush();
      offer(v[h].x);
      offer(v[h].y);
      offer(v[h].z);
      offer(v[h].w);
    }
  }
  if (queued > kQueue - 32) flush();
  offer(edge);
  flush();
}

// How often v stands in a list, by the whole CTA.
__device__ __forceinline__ int count_of(int v, const int32_t* list, int64_t n, int* s_exact) {
  __syncthreads();
  if (threadIdx.x == 0) *s_exact = 0;
  __syncthreads();
  int count = 0;
  for (int64_t j = threadIdx.x; j < n; j += kLogitThreads) count += list[j] == v;
  count = __reduce_add_sync(0xffffffffu, count);
  if ((threadIdx.x & 31) == 0) atomicAdd(s_exact, count);
  __syncthreads();
  return *s_exact;
}

// The places of the CTA's `mine` entries of a list's next kLogitThreads ones,
// in list order after `listed` earlier ones; adds their number to `listed`. One
// barrier; another one before s_warp is used again.
__device__ __forceinline__ int list_places(bool mine, int& listed, int* s_warp) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t m = __ballot_sync(0xffffffffu, mine);
  if (lane == 0) s_warp[warp] = __popc(m);
  __syncthreads();
  int before = listed;
#pragma unroll
  for (int w = 0; w < kLogitWarps; ++w) {
    before += w < warp ? s_warp[w] : 0;
    listed += s_warp[w];
  }
  return before + __popc(m & ((1u << lane) - 1));
}

// The met tokens of a share with more biases than are kept, which the pass has
// left alone, straight into out (a call of its own: inlined, its registers
// would be taken from the pass). kMet tokens at a time, first the sums of their
// biases, each token's in list order: the list goes by in pieces of
// kLogitThreads entries, and in each piece a token's first entry adds all of its
// own. (64 requests of 128000 tokens with 3000 biases each 117 us, with 20000
// 561; each biased token going through the list by itself: 230 and 44,000.)
template <typename T, typename OT>
__device__ __noinline__ void finish_many(const T* in, OT* out, int n, int v0, Penalty c,
                                         const uint32_t* mask, const int32_t* told, int64_t n_told,
                                         const int32_t* tokens, const float* values,
                                         int64_t n_biases, const uint16_t* s_bits, int* s_token,
                                         float* s_value, float* s_sum, int* s_warp, int* s_exact) {
  static_assert(kListed >= kLogitThreads, "a piece of the list");
  const int me = threadIdx.x;
  for (int lo = 0; lo < n; lo += kMet) {
    const int hi = min(lo + kMet, n);
    for (int k = lo + me; k < hi; k += kLogitThreads) s_sum[k - lo] = 0.f;
    int next = me < n_biases ? tokens[me] : -1;
    for (int64_t k = me; k - me < n_biases; k += kLogitThreads) {
      const unsigned at = (unsigned)next - (unsigned)(v0 + lo);
      const bool mine = at < (unsigned)(hi - lo);
      const float value = mine ? values[k] : 0.f;
      next = k + kLogitThreads < n_biases ? tokens[k + kLogitThreads] : -1;
      int total = 0;
      const int place = list_places(mine, total, s_warp);
      if (mine) s_token[place] = (int)at, s_value[place] = value;
      __syncthreads();
      if (me < total) {
        const int t = s_token[me];
        int j = 0;
        while (s_token[j] != t) ++j;
        if (j == me) {
          float sum = s_sum[t];
          for (; j < total; ++j)
            if (s_token[j] == t) sum += s_value[j];
          s_sum[t] = sum;
        }
      }
    }
    __syncthreads();
    const auto finish = [&](int k, uint32_t w, int64_t count) {
      float l = penalised(to_f32(in[k]), w & kSeen, count, c);
      if (w & kBiased) l += s_sum[k - lo];
      out[k] = from_f32<OT>(mask && !(mask[k / 32] >> (k % 32) & 1u) ? -INFINITY : l);
    };
    for (int k = lo + me; k < hi; k += kLogitThreads) {
      const uint32_t w = s_bits[k];
      if (w != 0 && (w & kCount) < kHeavy) finish(k, w, w & kCount);
    }
    if (n_told >= (int64_t)kHeavy)
      for (int k = lo; k < hi; ++k) {
        const uint32_t w = s_bits[k];
        if ((w & kCount) < kHeavy) continue;
        const int count = count_of(v0 + k, told, n_told, s_exact);
        if (me == 0) finish(k, w, count);
      }
    __syncthreads();
  }
}

// CTAs take (request, share of the vocabulary) pairs in turn; the next one's
// parameters come into registers early and, where logits are loaded element by
// element (VEC 1: the rows of out have other boundaries than those of the
// logits), its logits into L2: 256 x 50257 fp32 41 us, 47 without. Whole
// vectors have enough under way themselves: 256 x 128000 75 us without, 76
// with. A token's bits of the table are cleared as it is put in place.
template <typename T, typename OT, int VEC>
__global__ void __launch_bounds__(kLogitThreads, kLogitPerSm) logits_rows(LogitArgs a) {
  extern __shared__ __align__(16) uint32_t s_word[];  // a.share / 2 words, two tokens each
  __shared__ uint16_t s_met[kMet];
  __shared__ float s_result[kMet];
  __shared__ int s_token[kListed];
  __shared__ float s_value[kListed];
  __shared__ int s_warp[kLogitWarps];
  __shared__ uint16_t s_queue[kLogitWarps][kQueue];
  __shared__ int s_n, s_exact;  // met tokens; an exact count
  constexpr int kBatch = VEC == 1 ? 8 : 4;  // vectors under way per thread
  const spmv_logits& p = a.l;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, me = threadIdx.x;
  const int64_t jobs = (int64_t)p.n_requests * a.shares;
  const auto ask_logits = [&](int64_t i, int v0) {
    if (VEC == 1 && me == 0)
      prefetch_bulk(static_cast<const T*>(p.logits) + i * p.stride + v0,
                    min(a.share, p.vocab - v0) * (int64_t)sizeof(T));
  };
  const auto bits_of = [&](int k) { return s_word[k >> 1] >> (16 * (k & 1)) & 0xffffu; };
  int64_t i = blockIdx.x / (unsigned)a.shares;
  int v0 = (int)(blockIdx.x % (unsigned)a.shares) * a.share;
  const int64_t step_i = gridDim.x / (unsigned)a.shares;
  // (the end of a row's last share, and a step beyond it, may pass 31 bits)
  const unsigned step_v = gridDim.x % (unsigned)a.shares * (unsigned)a.share;
  const unsigned wrap = (unsigned)a.shares * (unsigned)a.share;
  ask_logits(i, v0);
  Request next;
  next.load(p, i);
  const auto clear_table = [&] {
    for (int k = 4 * me; k < a.share / 2; k += 4 * kLogitThreads)
      *reinterpret_cast<uint4*>(s_word + k) = make_uint4(0, 0, 0, 0);
  };
  clear_table();
  if (me == 0) s_n = 0;
  __syncthreads();

  for (int64_t id = blockIdx.x; id < jobs; id += gridDim.x) {
    const int n = min(a.share, p.vocab - v0);
    const T* in = static_cast<const T*>(p.logits) + i * p.stride + v0;
    OT* out = static_cast<OT*>(p.out) + i * p.out_stride + v0;
    Request q = next;
    q.settle(p);
    int64_t next_i = i + step_i;
    unsigned next_v = (unsigned)v0 + step_v;
    if (next_v >= wrap) next_v -= wrap, ++next_i;
    const bool more = id + gridDim.x < jobs;
    if (more) next.load(p, next_i);
    const uint32_t* mask = q.mask_row >= 0 ? p.mask + q.mask_row * p.mask_stride + v0 / 32 : nullptr;

    // count the lists; who first meets a token puts it on the list of met ones
    // (in whatever order: each is finished by itself)
    const auto mark = [&](int k, uint32_t how) {
      return (atomicOr(s_word + (k >> 1), how << (16 * (k & 1))) >> (16 * (k & 1)) & 0xffffu) == 0;
    };
    const auto seen = [&](int k) {  // (frequent tokens once: atomics of one address queue up)
      return !(bits_of(k) & kSeen) && mark(k, kSeen);
    };
    const auto told = [&](int k) {
      return (bits_of(k) & kCount) < kHeavy &&
             (atomicAdd(s_word + (k >> 1), 1u << (16 * (k & 1))) >> (16 * (k & 1)) & 0xffffu) == 0;
    };
    for_entries(p.prompt_tokens, q.p0, q.p1, v0, n, s_queue[warp], &s_n, s_met, seen);
    for_entries(p.output_tokens, q.o0, q.o1, v0, n, s_queue[warp], &s_n, s_met, told);
    if (more) ask_logits(next_i, (int)next_v);
    // biases of this CTA's tokens, compacted in list order
    int listed = 0;
    for (int64_t k = q.b0; k < q.b1; k += kLogitThreads) {
      const bool on = k + me < q.b1;
      const int v = on ? p.bias_tokens[k + me] : -1;
      const float value = on ? p.bias_values[k + me] : 0.f;
      const bool mine = v >= v0 && v < v0 + n;
      list_met(mine && mark(v - v0, kBiased), v - v0, &s_n, s_met);
      const int place = list_places(mine, listed, s_warp);
      if (mine && place < kListed) {
        s_token[place] = v;
        s_value[place] = value;
      }
      if (k + kLogitThreads < q.b1) __syncthreads();
    }
    // (told with the count: a branch on `listed` itself makes the compiler spill
    // 260 bytes, and 256 x 128000 take 103 us for 74)
    if (me == 0 && listed > kListed) atomicAdd(&s_n, kMany);
    __syncthreads();
    const int met = s_n;
    // A pair without met tokens has no further barrier, and a warp that is done
    // with its part of the pass would raise s_n for the next pair: not before
    // every warp has read it.
    if (met == 0) __syncthreads();
    const bool kept = met <= kMet;  // on the list, all of them
    // a met token's result
    const auto result = [&](int k, uint32_t w, int64_t count) {
      float l = penalised(to_f32(in[k]), w & kSeen, count, q.c);
      if (w & kBiased) {
        float sum = 0.f;
        for (int j = 0; j < listed; ++j)
          if (s_token[j] == v0 + k) sum += s_value[j];
        l += sum;
      }
      return mask && !(mask[k / 32] >> (k % 32) & 1u) ? -INFINITY : l;
    };
    if (met > 0 && met < kMany) {
      // Results of the met tokens: into the list's places or, where there are
      // more than it holds, straight into out, which the pass then leaves
      // alone there. (out may be the logits themselves: they are read first.
      // Shares with more than kListed biases come after the pass.)
      for (int e = me; e < (kept ? met : n); e += kLogitThreads) {
        const int k = kept ? s_met[e] : e;
        const uint32_t w = bits_of(k);
        if (w == 0 || (w & kCount) >= kHeavy) continue;
        const float l = result(k, w, w & kCount);
        if (kept)
          s_result[e] = l;
        else
          out[k] = from_f32<OT>(l);
      }
      if (q.o1 - q.o0 >= (int64_t)kHeavy) {  // counts past the table's: by the whole CTA
        for (int e = 0; e < (kept ? met : n); ++e) {
          const int k = kept ? s_met[e] : e;
          const uint32_t w = bits_of(k);
          if ((w & kCount) < kHeavy) continue;
          const int count = count_of(v0 + k, p.output_tokens + q.o0, q.o1 - q.o0, &s_exact);
          if (me == 0) {
            const float l = result(k, w, count);
            if (kept)
              s_result[e] = l;
            else
              out[k] = from_f32<OT>(l);
          }
        }
      }
      __syncthreads();
    }
    // Whole vectors from the row's first boundary on (out's is at the same
    // token), single tokens before and after them. (256 x 50257 fp32: 35 us,
    // element by element 41.)
    int lead = 0, whole = n;
    if constexpr (VEC > 1) {
      lead = min((int)(0u - (unsigned)(reinterpret_cast<uintptr_t>(in) / sizeof(T))) & (VEC - 1), n);
      whole = lead + (n - lead) / VEC * VEC;
      const int k = me < VEC ? (me < lead ? me : n) : whole + me - VEC;
      if (me < 2 * VEC && k < n && (kept || bits_of(k) == 0))
        out[k] = from_f32<OT>(!mask || mask[k / 32] >> (k % 32) & 1u ? to_f32(in[k]) : -INFINITY);
    }
    for (int base = lead + VEC * me; base < whole; base += kBatch * VEC * kLogitThreads) {
      Pack<T, VEC> v[kBatch];
      uint32_t bits[kBatch];  // of the VEC tokens from k on
#pragma unroll
      for (int h = 0; h < kBatch; ++h) {
        const int k = base + h * VEC * kLogitThreads;
        if (k < whole) v[h] = load_pack<T, VEC>(in + k, true);
      }
#pragma unroll
      for (int h = 0; h < kBatch; ++h) {
        const int k = base + h * VEC * kLogitThreads;
        bits[h] = 0xffffffffu;
        if (mask && k < whole)
          bits[h] = __funnelshift_r(__ldg(mask + k / 32), __ldg(mask + (k + VEC - 1) / 32), k % 32);
      }
#pragma unroll
      for (int h = 0; h < kBatch; ++h) {
        const int k = base + h * VEC * kLogitThreads;
        Pack<OT, VEC> r;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          r.v[e] = from_f32<OT>(bits[h] >> e & 1 ? to_f32(v[h].v[e]) : -INFINITY);
        if (k >= whole) break;
        if (kept) {
          store_pack<OT, VEC>(out + k, r);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e)
            if (bits_of(k + e) == 0) out[k + e] = r.v[e];
        }
      }
    }
    if (met > 0) {
      __syncthreads();
      if (kept) {
        for (int e = me; e < met; e += kLogitThreads) {
          out[s_met[e]] = from_f32<OT>(s_result[e]);
          reinterpret_cast<uint16_t*>(s_word)[s_met[e]] = 0;
        }
      } else {
        if (met >= kMany)
          finish_many(in, out, n, v0, q.c, mask, p.output_tokens + q.o0, q.o1 - q.o0,
                      p.bias_tokens + q.b0, p.bias_values + q.b0, q.b1 - q.b0,
                      reinterpret_cast<const uint16_t*>(s_word), s_token, s_value, s_result,
                      s_warp, &s_exact);
        clear_table();
      }
      if (me == 0) s_n = 0;
      __syncthreads();
    }
    i = next_i;
    v0 = (int)next_v;
  }
}

template <typename T, typename OT>
spmv_status launch_logits(const spmv_logits& p, cudaStream_t st) {
  LogitArgs a{};
  a.l = p;
  // Every list is read once for each share, so shares are large; but CTAs
  // should be done together. Of the counts that a table allows, up to twice the
  // least: the one with the least of rounds x (a round's lists, some 15,000
  // tokens' time, and its tokens). (256 x 128000 fp32: 75 us; 97 where the
  // lists count for nothing. Tables for shares of 16384 tokens: 80.)
  const int least = (int)((p.vocab + (int64_t)kShare - 1) / kShare);
  int64_t best = INT64_MAX;
  for (int s = least; s <= 2 * least; ++s) {
    const int64_t rounds = ((int64_t)p.n_requests * s + kWave - 1) / kWave;
    const int64_t cost = rounds * (15000 + p.vocab / s);
    if (cost < best) best = cost, a.shares = s;
  }
  // few requests: shares for every SM's first two CTAs (37 x 50257 bf16: 12.9
  // us, for all three 14.5, for the first 14.4)
  const int64_t spread = 2 * 152 / p.n_requests, most = (p.vocab + kLeastShare - 1ll) / kLeastShare;
  if (a.shares < spread && a.shares < most) a.shares = (int)(spread < most ? spread : most);
  a.share = (int)(((int64_t)p.vocab + a.shares - 1) / a.shares + 31) / 32 * 32;
  a.shares = (int)(((int64_t)p.vocab + a.share - 1) / a.share);
  // Vectors of 16 bytes of out, where each row's boundaries are at the same
  // tokens in both (256 x 128000 bf16 to fp32: 68 us; 16 bytes of the logits:
  // 84).
  constexpr int kVec = 16 / (int)sizeof(OT);
  const bool vec = (reinterpret_cast<uintptr_t>(p.logits) / sizeof(T) -
                    reinterpret_cast<uintptr_t>(p.out) / sizeof(OT)) % kVec == 0 &&
                   (p.n_requests == 1 || (p.stride - p.out_stride) % kVec == 0);
  const void* fn = vec ? reinterpret_cast<const void*>(&logits_rows<T, OT, kVec>)
                       : reinterpret_cast<const void*>(&logits_rows<T, OT, 1>);
  const size_t smem = (size_t)a.share * 2;
  if (!allow_smem(fn, smem)) return SPMV_ERR_CUDA;
  const int64_t jobs = (int64_t)p.n_requests * a.shares;
  void* args[] = {&a};
  return status_of(cudaLaunchKernel(fn, dim3((unsigned)(jobs < kWave ? jobs : kWave)),
                                    dim3(kLogitThreads), args, smem, st));
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
