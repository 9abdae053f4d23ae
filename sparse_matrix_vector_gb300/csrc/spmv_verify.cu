// Verification of drafted tokens (spmv_verify_drafts). With p the target's and
// q the drafter's probabilities at a position, the drafted token x is accepted
// where u q(x) < p(x); the request's last token is drawn from what p has over
// q at its first rejected position, or from p behind its last draft.
//
// Two launches. verify_rows is bound by reading every row of logits once:
// largest logit and sum of exponentials of a share of a row, or its largest
// token for greedy requests. verify_pick, a cluster per request, joins the
// shares, walks through the request's drafts and draws the token; it reads
// one or two rows again, mostly from L2.
//
// Whole numbers leave no room for rounding: which token a random number falls
// on is decided by running sums over the vocabulary whose borders may be
// nearer to each other than fp32's roundings. So the row that a token is drawn
// from is summed in pairs of fp32, and so are the rows of a draft whose test
// is too near to call in fp32 (within kNear).
#include <cooperative_groups.h>

#include <climits>

#include "spmv_device.cuh"
#include "spmv_duo.cuh"
#include "spmv_softmax.cuh"
#include "spmv_types.cuh"

namespace spmv {
namespace {

namespace cg = cooperative_groups;

constexpr int kRowThreads = 256;
constexpr int kRowAtOnce = 4;
constexpr int kPickThreads = 512, kPickWarps = kPickThreads / 32;
constexpr int kMaxCluster = 8;
constexpr float kNear = 1e-4f;
constexpr int kNone = INT_MAX;

struct Part {  // of a share of a row
  float m, s;
  int best;    // the first token with the largest logit; kNone: nothing above minus infinity
  int unused;
};

struct VerifyArgs {
  int n, d, vocab;
  const void* target;
  int64_t target_stride;
  const void* draft;
  int64_t draft_stride;
  const int32_t* tokens;
  const int64_t* offsets;
  const float *accept_u, *sample_u, *temperature;
  int32_t *out, *accepted;
  Part* parts;  // [target rows, then draft rows][shares]
  int shares, share;
};

// NaN counts as minus infinity, plus infinity as the largest number.
__device__ __forceinline__ float cleaned(float v) { return v == v ? fminf(v, FLT_MAX) : -INFINITY; }

// 0: greedy
__device__ __forceinline__ float temperature_of(const VerifyArgs& a, int i) {
  const float t = a.temperature ? a.temperature[i] : 1.f;
  return t > 0.f ? fminf(fmaxf(t, 1e-30f), 1e30f) : 0.f;
}
__device__ __forceinline__ float scale_of(float t) { return (float)(1.4426950408889634 / (double)t); }

__device__ __forceinline__ int64_t offset_at(const VerifyArgs& a, int i) {
  const int64_t o = a.offsets[i];
  return o < 0 ? 0 : o > a.d ? a.d : o;
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads, 4) verify_rows(VerifyArgs a) {
  __shared__ MaxSum s_red[kRowThreads / 32];
  __shared__ int s_best[kRowThreads / 32];
  const int me = threadIdx.x;
  const int64_t slot = blockIdx.x / a.shares;
  const int rank = (int)(blockIdx.x - slot * a.shares);
  const bool of_draft = slot >= a.d + a.n;
  const int64_t r = of_draft ? slot - (a.d + a.n) : slot;
  // the row's request: the last one whose rows begin at or before it
  int before = 0;
  for (int b = 0; b < a.n; b += kRowThreads) {
    const int i = b + me;
    before += __syncthreads_count(i < a.n && offset_at(a, i) + (of_draft ? 0 : i) <= r);
  }
  if (before == 0 || r >= offset_at(a, a.n) + (of_draft ? 0 : a.n)) return;  // no request's
  const float t = temperature_of(a, before - 1);
  if (of_draft && t == 0.f) return;
  const T* row = of_draft ? static_cast<const T*>(a.draft) + r * a.draft_stride
                          : static_cast<const T*>(a.target) + r * a.target_stride;
  const int64_t lo = (int64_t)rank * a.share;
  const int n = (int)min((int64_t)a.share, (int64_t)a.vocab - lo);
  row += lo;
  Part out{-FLT_MAX, 0.f, kNone, 0};
  if (t == 0.f) {
    float m = -INFINITY;
    int at = kNone;
    for_units<kRowThreads, kRowAtOnce>(row, n, [&](int v0, float (&v)[kUnit]) {
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kUnit; ++k) top = fmaxf(top, v[k]);
      if (top > m || (top == m && top > -INFINITY && v0 < at)) m = top, at = v0;
    });
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o);
      const int at2 = __shfl_xor_sync(0xffffffffu, at, o);
      if (m2 > m || (m2 == m && at2 < at)) m = m2, at = at2;
    }
    if ((me & 31) == 0) s_red[me >> 5].m = m, s_best[me >> 5] = at;
    __syncthreads();
    if (me == 0) {
      for (int w = 1; w < kRowThreads / 32; ++w)
        if (s_red[w].m > m || (s_red[w].m == m && s_best[w] < at)) m = s_red[w].m, at = s_best[w];
      if (at != kNone) {
        while (to_f32(row[at]) != m) ++at;  // (within a unit: one of its tokens is the largest)
        at += (int)lo;
      }
      out.m = m;
      out.best = at;
    }
  } else {
    const float c = scale_of(t);
    MaxSum x = MaxSum::none();
    for_units<kRowThreads, kRowAtOnce>(row, n, [&](int, float (&v)[kUnit]) { x.add(v, c); });
    x = join_cta<kRowThreads>(x, c, s_red);
    if (!(x.s == x.s) || x.m > FLT_MAX) {  // NaN or plus infinity in the share: again, cleaned
      __syncthreads();
      x = MaxSum::none();
      for_units<kRowThreads, kRowAtOnce>(row, n, [&](int, float (&v)[kUnit]) {
#pragma unroll
        for (int k = 0; k < kUnit; ++k) v[k] = cleaned(v[k]);
        x.add(v, c);
      });
      x = join_cta<kRowThreads>(x, c, s_red);
    }
    out.m = x.m;
    out.s = x.s;
  }
  if (me == 0) a.parts[slot * a.shares + rank] = out;
}

// A row's shares joined, by one warp (the same in all lanes).
__device__ __forceinline__ Part join_row(const VerifyArgs& a, int64_t slot, float c) {
  const int lane = threadIdx.x & 31;
  MaxSum x = MaxSum::none();
  float m = -INFINITY;
  int at = kNone;
  for (int k = lane; k < a.shares; k += 32) {
    const Part p = a.parts[slot * a.shares + k];
    x.join({p.m, p.s}, c);
    if (p.m > m || (p.m == m && p.best < at)) m = p.m, at = p.best;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const MaxSum y{__shfl_xor_sync(0xffffffffu, x.m, o), __shfl_xor_sync(0xffffffffu, x.s, o)};
    const float to = fmaxf(x.m, y.m);
    x.s = x.s * exp2_fast((x.m - to) * c) + y.s * exp2_fast((y.m - to) * c);
    x.m = to;
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o);
    const int at2 = __shfl_xor_sync(0xffffffffu, at, o);
    if (m2 > m || (m2 == m && at2 < at)) m = m2, at = at2;
  }
  return Part{x.m, x.s, at, 0};
}

struct Pick {  // a CTA's shared memory
  float2 roots[64];
  double seg[2][kPickWarps];  // sums of its warps' segments: the target's or what is left of it, the drafter's
  double all[2][kMaxCluster * kPickWarps];
  double sub[kPickWarps];
  int last[kPickWarps];
  float p_m[kPickWarps], p_s[kPickWarps], q_m[kPickWarps], q_s[kPickWarps];
  int best[kPickWarps], verdict[kPickWarps];
  int any_last;
  int where;
};

// 2^((l - m) c) of a row's logits, in pairs.
struct RowExp {
  float m;
  Duo c;
  const float2* roots;
  __device__ __forceinline__ Duo operator()(float l) const {
    return duo_exp2(duo_mul(two_sum(cleaned(l), -m), c), roots);
  }
};

__device__ __forceinline__ double sum_lanes(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// What a token has to be drawn by: the target's exponentials, less those of
// the drafter times alpha where a draft was rejected, less the draft itself
// where it carries no probabilities.
template <typename T>
struct Weight {
  const T* target;
  const T* draft;  // null: none to take off
  RowExp ep, eq;
  Duo alpha;
  int skip;        // a token without weight; -1: none
  __device__ __forceinline__ Duo operator()(int v) const {
    Duo w = ep(to_f32(target[v]));
    if (draft) {
      const Duo t = duo_mul(eq(to_f32(draft[v])), alpha);
      w = duo_add(w, {-t.h, -t.l});
    }
    if (v == skip || !(w.h > 0.f)) w = {0.f, 0.f};
    return w;
  }
};

// Sum over tokens [lo, hi) by a warp, and the last of them with a weight (-1: none).
template <typename W>
__device__ __forceinline__ double sum_range(const W& w, int64_t lo, int64_t hi, int* last) {
  Duo s{0.f, 0.f};
  int end = -1;
#pragma unroll 4
  for (int64_t v = lo + (threadIdx.x & 31); v < hi; v += 32) {
    const Duo e = w((int)v);
    s = duo_add(s, e);
    if (e.h > 0.f) end = (int)v;
  }
  *last = __reduce_max_sync(0xffffffffu, end);
  return sum_lanes(to_f64(s));
}

template <typename T>
__global__ void __launch_bounds__(kPickThreads) verify_pick(VerifyArgs a) {
  __shared__ Pick s;
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int i = blockIdx.x / ctas, me = threadIdx.x, warp = me >> 5, lane = me & 31;
  if (me < 64) s.roots[me] = kRoots[me];
  pdl_wait();
  const int64_t off = offset_at(a, i);
  const int64_t end = offset_at(a, i + 1);
  const int len = end > off ? (int)(end - off) : 0;
  const float t = temperature_of(a, i);
  const bool greedy = t == 0.f;
  const float c = greedy ? 1.f : scale_of(t);
  const Duo c2 = duo_of(greedy ? 1.0 : 1.4426950408889634073599 / (double)t);
  const int64_t first = off + i;  // the request's first row of the target
  // segments of the vocabulary, one per warp of the cluster
  const int64_t seg = ((int64_t)a.vocab + ctas * kPickWarps - 1) / (ctas * kPickWarps);
  const int64_t lo = min((int64_t)a.vocab, (rank * kPickWarps + warp) * seg);
  const int64_t hi = min((int64_t)a.vocab, lo + seg);
  const auto target_row = [&](int j) { return static_cast<const T*>(a.target) + (first + j) * a.target_stride; };
  const auto draft_row = [&](int j) { return static_cast<const T*>(a.draft) + (off + j) * a.draft_stride; };
  // both rows' sums at position j, in pairs; the same in the whole cluster
  const auto exact_sums = [&](int j, float pm, float qm, bool with_draft, double* sp, double* sq) {
    int none;
    const Weight<T> wp{target_row(j), nullptr, {pm, c2, s.roots}, {}, {}, -1};
    const double p = sum_range(wp, lo, hi, &none);
    double q = 0;
    if (with_draft) {
      const Weight<T> wq{draft_row(j), nullptr, {qm, c2, s.roots}, {}, {}, -1};
      q = sum_range(wq, lo, hi, &none);
    }
    if (lane == 0) s.seg[0][warp] = p, s.seg[1][warp] = q;
    cluster.sync();
    for (int k = me; k < ctas * kPickWarps; k += kPickThreads) {
      const Pick* other = cluster.map_shared_rank(&s, k / kPickWarps);
      s.all[0][k] = other->seg[0][k % kPickWarps];
      s.all[1][k] = other->seg[1][k % kPickWarps];
    }
    cluster.sync();
    double tp = 0, tq = 0;
    for (int k = lane; k < ctas * kPickWarps; k += 32) tp += s.all[0][k], tq += s.all[1][k];
    *sp = sum_lanes(tp);
    *sq = sum_lanes(tq);
  };
  // the probability, times the sum, of one token in fp64 (0 where fp32 has none)
  const auto exact_exp = [&](float l, float m) {
    l = cleaned(l);
    return (l - m) * c < -126.f ? 0.0 : exp(((double)l - (double)m) / (double)t);
  };

  // the first rejected draft, kPickWarps at a time
  int taken = len, x = -1;
  float pm = 0.f, qm = 0.f;
  int best = kNone;
  bool with_draft = false;
  for (int j0 = 0; j0 <= len && taken == len; j0 += kPickWarps) {
    const int j = j0 + warp;
    __syncthreads();
    if (j <= len) {
      const Part p = join_row(a, first + j, c);
      Part q{0.f, 1.f, 0, 0};
      int verdict = 0;  // 0 accepted, 1 rejected, 2 too near to call
      if (j < len) {
        const int id = a.tokens[off + j];
        const bool valid = (unsigned)id < (unsigned)a.vocab;
        if (a.draft && !greedy) q = join_row(a, (int64_t)a.d + a.n + off + j, c);
        if (greedy) {
          verdict = !(valid && id == p.best);
        } else if (!valid) {
          verdict = 1;
        } else {
          const float l = cleaned(to_f32(target_row(j)[id]));
          const float u = a.accept_u[off + j];
          const float pe = p.s > 0.f ? exp2_fast((l - p.m) * c) / p.s : 0.f;
          float qe = 1.f;
          if (a.draft) qe = q.s > 0.f ? exp2_fast((cleaned(to_f32(draft_row(j)[id])) - q.m) * c) / q.s : 0.f;
          const float uq = u * qe;
          verdict = !(uq < pe);
          if (fabsf(uq - pe) <= kNear * fmaxf(uq, pe) && pe > 0.f) verdict = 2;
        }
      }
      if (lane == 0) {
        s.p_m[warp] = p.m, s.q_m[warp] = q.m, s.q_s[warp] = q.s, s.best[warp] = p.best;
        s.verdict[warp] = verdict;
      }
    }
    __syncthreads();
    for (int k = 0; k < kPickWarps && j0 + k <= len; ++k) {
      pm = s.p_m[k], qm = s.q_m[k], best = s.best[k];
      with_draft = a.draft && s.q_s[k] > 0.f;
      int verdict = s.verdict[k];
      if (verdict == 2) {
        double sp, sq;
        exact_sums(j0 + k, pm, qm, a.draft != nullptr, &sp, &sq);
        const int id = a.tokens[off + j0 + k];
        const double pe = exact_exp(to_f32(target_row(j0 + k)[id]), pm);
        const double u = (double)a.accept_u[off + j0 + k];
        const bool ok = a.draft ? u * exact_exp(to_f32(draft_row(j0 + k)[id]), qm) * sp < pe * sq : u * sp < pe;
        verdict = !ok;
      }
      if (j0 + k < len && verdict) {
        taken = j0 + k;
        break;
      }
    }
  }
  if (taken < len) {
    const int id = a.tokens[off + taken];
    x = (unsigned)id < (unsigned)a.vocab ? id : -1;
  }
  // the accepted drafts, and nothing behind the last token
  if (rank == 0) {
    for (int j = me; j <= len; j += kPickThreads)
      if (j != taken) a.out[first + j] = j < taken ? a.tokens[off + j] : -1;
    if (me == 0) a.accepted[i] = taken;
  }
  if (greedy) {
    if (rank == 0 && me == 0) a.out[first + taken] = best == kNone ? -1 : best;
    return;
  }

  // the last token: the first whose running sum passes the random number's
  // share of the whole
  const bool residual = taken < len;
  const bool take_off = residual && a.draft && with_draft;
  double sp, sq;
  exact_sums(taken, pm, qm, take_off, &sp, &sq);
  Weight<T> w{target_row(taken), nullptr, {pm, c2, s.roots}, {qm, c2, s.roots}, {0.f, 0.f}, -1};
  double total = sp;
  if (residual && (take_off || (!a.draft && x >= 0))) {
    if (take_off) {
      w.draft = draft_row(taken);
      w.alpha = duo_of(sp / sq);
    } else {
      w.skip = x;
    }
    int none;
    const double mine = sum_range(w, lo, hi, &none);
    if (lane == 0) s.seg[0][warp] = mine;
    cluster.sync();
    for (int k = me; k < ctas * kPickWarps; k += kPickThreads)
      s.all[1][k] = cluster.map_shared_rank(&s, k / kPickWarps)->seg[0][k % kPickWarps];
    cluster.sync();
    double sum = 0;
    for (int k = lane; k < ctas * kPickWarps; k += 32) sum += s.all[1][k];
    sum = sum_lanes(sum);
    if (sum > 0) {
      total = sum;
      for (int k = me; k < ctas * kPickWarps; k += kPickThreads) s.all[0][k] = s.all[1][k];
    } else {  // nothing is left (p = q): from p
      w.draft = nullptr;
      w.skip = -1;
    }
    __syncthreads();
  }
  const double goal = (double)a.sample_u[i] * total;
  // the segment: lane l holds segments [l * per, (l + 1) * per)
  if (warp == 0) {
    const int n = ctas * kPickWarps, per = (n + 31) / 32;
    double sum = 0;
    for (int k = 0; k < per; ++k)
      if (lane * per + k < n) sum += s.all[0][lane * per + k];
    double upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    double run = __shfl_up_sync(0xffffffffu, upto, 1);
    if (lane == 0) run = 0;
    int at = kNone, last = -1;
    double base = 0;
    for (int k = 0; k < per; ++k)
      if (lane * per + k < n) {
        const double v = s.all[0][lane * per + k];
        if (v > 0) last = lane * per + k;
        if (at == kNone && v > 0 && run + v > goal) at = lane * per + k, base = run;
        run += v;
      }
    const int found = __reduce_min_sync(0xffffffffu, at), end_seg = __reduce_max_sync(0xffffffffu, last);
    const uint32_t who = __ballot_sync(0xffffffffu, at == found && at != kNone);
    base = __shfl_sync(0xffffffffu, base, who ? __ffs(who) - 1 : 0);
    if (lane == 0) {
      s.where = found != kNone ? found : end_seg;
      s.sub[0] = found != kNone ? base : INFINITY;  // (past the end: the last token with a weight)
    }
  }
  __syncthreads();
  const int where = s.where;
  double run = s.sub[0];
  __syncthreads();
  if (where < 0) {  // a row without any token
    if (rank == 0 && me == 0) a.out[first + taken] = -1;
    return;
  }
  if (where / kPickWarps != rank) return;
  // its warps' parts of the segment, then the part's tokens
  const int64_t s_lo = min((int64_t)a.vocab, where * seg), s_hi = min((int64_t)a.vocab, s_lo + seg);
  const int64_t part = (seg + kPickWarps - 1) / kPickWarps;
  const int64_t p_lo = min(s_hi, s_lo + warp * part), p_hi = min(s_hi, p_lo + part);
  int last;
  const double mine = sum_range(w, p_lo, p_hi, &last);
  if (lane == 0) s.sub[warp] = mine, s.last[warp] = last;
  __syncthreads();
  int chosen = -1, fallback = -1;
  double begin = run;
  for (int k = 0; k < kPickWarps; ++k) {
    const double v = s.sub[k];
    if (s.last[k] >= 0) fallback = s.last[k];
    if (chosen < 0 && v > 0 && run + v > goal && run <= goal) chosen = k, begin = run;
    if (chosen < 0 && v > 0 && run > goal && run < INFINITY) chosen = k, begin = run;
    run += v;
  }
  if (chosen < 0) {
    if (me == 0) a.out[first + taken] = fallback;
    return;
  }
  if (warp != chosen) return;
  int token = -1;
  for (int64_t v0 = p_lo; v0 < p_hi && token < 0; v0 += 32) {
    const int64_t v = v0 + lane;
    const double e = v < p_hi ? to_f64(w((int)v)) : 0;
    double upto = e;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    const uint32_t over = __ballot_sync(0xffffffffu, e > 0 && begin + upto > goal);
    if (over) token = (int)v0 + __ffs(over) - 1;
    begin += __shfl_sync(0xffffffffu, upto, 31);
  }
  if (lane == 0) a.out[first + taken] = token >= 0 ? token : s.last[warp];
}

constexpr int kWave = 4 * 152;  // CTAs that the device's SMs hold at a time

struct Split {
  int shares, share;
};

// Shares of a row: at most 32768 tokens each (a CTA's time, some 10 us, is
// what the last wave of CTAs may leave unused), more of them where rows are
// few, down to 1024 tokens.
Split split_of(int64_t rows, int vocab) {
  const int64_t least = (vocab + 32767ll) / 32768, most = (vocab + 1023ll) / 1024;
  int64_t s = rows > 0 ? kWave / rows : 1;
  s = s > most ? most : s;
  s = s < least ? least : s;
  const int64_t share = ((vocab + s - 1) / s + 63) / 64 * 64;
  return {(int)((vocab + share - 1) / share), (int)share};
}

int64_t rows_of(int64_t n, int64_t d, bool with_draft) { return n + d + (with_draft ? d : 0); }

// Rows that a call may have, and jobs of the first launch.
bool too_many(int64_t rows, int vocab) {
  return rows > (1 << 24) || rows * split_of(rows, vocab).shares > INT_MAX;
}

template <typename T>
spmv_status launch_verify(VerifyArgs& a, cudaStream_t st) {
  const int64_t rows = rows_of(a.n, a.d, a.draft != nullptr);
  const spmv_status s = launch(verify_rows<T>, dim3((unsigned)(rows * a.shares)), kRowThreads, 0, st, a);
  if (s != SPMV_OK) return s;
  int ctas = kMaxCluster;
  while (ctas > 1 && (int64_t)ctas * a.n > 2 * 152) ctas /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.n * ctas));
  cfg.blockDim = dim3(kPickThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  void* args[] = {&a};
  return status_of(cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(&verify_pick<T>), args));
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" int64_t spmv_verify_workspace(int32_t n_requests, int32_t n_drafts, int32_t vocab) {
  if (n_requests < 1 || n_drafts < 0 || vocab < 1 || vocab > INT_MAX - 4096 ||
      too_many(rows_of(n_requests, n_drafts, true), vocab))
    return 0;
  // (for either number of rows)
  int64_t most = 0;
  for (int k = 0; k < 2; ++k) {
    const int64_t rows = rows_of(n_requests, n_drafts, k);
    const int64_t bytes = rows * split_of(rows, vocab).shares * (int64_t)sizeof(Part);
    most = bytes > most ? bytes : most;
  }
  return most;
}

extern "C" spmv_status spmv_verify_drafts(int32_t n_requests, int32_t n_drafts, int32_t vocab,
                                          spmv_dtype dtype, const void* target, int64_t target_stride,
                                          const void* draft, int64_t draft_stride,
                                          const int32_t* draft_tokens, const int64_t* offsets,
                                          const float* accept_uniforms, const float* sample_uniforms,
                                          const float* temperature, int32_t* tokens, int32_t* accepted,
                                          void* workspace, int64_t workspace_bytes, void* stream) {
  if (n_requests < 0 || n_drafts < 0 || vocab < 1 || !op_dtype(dtype)) return SPMV_ERR_INVALID_ARG;
  if (vocab > INT_MAX - 4096 || too_many(rows_of(n_requests, n_drafts, true), vocab)) return SPMV_ERR_TOO_LARGE;
  const int64_t rows = (int64_t)n_requests + n_drafts, xs = op_dtype_size(dtype);
  if (n_requests == 0) return SPMV_OK;
  if (!matrix_ok(target, rows, vocab, target_stride, xs, false) ||
      (draft && !matrix_ok(draft, n_drafts, vocab, draft_stride, xs, false)) || !offsets ||
      !sample_uniforms || !tokens || !accepted || (n_drafts > 0 && (!draft_tokens || !accept_uniforms)) ||
      !aligned_to(draft_tokens, 4) || !aligned_to(offsets, 8) || !aligned_to(accept_uniforms, 4) ||
      !aligned_to(sample_uniforms, 4) || !aligned_to(temperature, 4) || !aligned_to(tokens, 4) ||
      !aligned_to(accepted, 4) || !aligned_to(workspace, 16))
    return SPMV_ERR_INVALID_ARG;
  const int64_t need = spmv_verify_workspace(n_requests, n_drafts, vocab);
  if (!workspace || workspace_bytes < need) return SPMV_ERR_INVALID_ARG;
  struct Span {
    const void* p;
    int64_t rows, cols, stride, size;
  };
  const Span outs[] = {{tokens, 1, rows, rows, 4}, {accepted, 1, n_requests, n_requests, 4}, {workspace, 1, need, need, 1}};
  const Span ins[] = {{target, rows, vocab, target_stride, xs},
                      {draft, n_drafts, vocab, draft_stride, xs},
                      {draft_tokens, 1, n_drafts, n_drafts, 4},
                      {offsets, 1, n_requests + 1ll, n_requests + 1ll, 8},
                      {accept_uniforms, 1, n_drafts, n_drafts, 4},
                      {sample_uniforms, 1, n_requests, n_requests, 4},
                      {temperature, 1, n_requests, n_requests, 4}};
  const auto meet = [](const Span& p, const Span& q) {
    return spans_overlap(p.p, p.rows, p.cols, p.stride, p.size, q.p, q.rows, q.cols, q.stride, q.size);
  };
  for (const Span& o : outs)
    for (const Span& in : ins)
      if (meet(o, in)) return SPMV_ERR_INVALID_ARG;
  if (meet(outs[0], outs[1]) || meet(outs[0], outs[2]) || meet(outs[1], outs[2])) return SPMV_ERR_INVALID_ARG;
  VerifyArgs a{};
  a.n = n_requests, a.d = n_drafts, a.vocab = vocab;
  a.target = target, a.target_stride = target_stride;
  a.draft = n_drafts > 0 ? draft : nullptr, a.draft_stride = draft_stride;
  a.tokens = draft_tokens, a.offsets = offsets;
  a.accept_u = accept_uniforms, a.sample_u = sample_uniforms, a.temperature = temperature;
  a.out = tokens, a.accepted = accepted, a.parts = static_cast<Part*>(workspace);
  const Split split = split_of(rows_of(a.n, a.d, a.draft != nullptr), vocab);
  a.shares = split.shares, a.share = split.share;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SPMV_F32) return launch_verify<float>(a, st);
  return dtype == SPMV_F16 ? launch_verify<__half>(a, st) : launch_verify<__nv_bfloat16>(a, st);
}
