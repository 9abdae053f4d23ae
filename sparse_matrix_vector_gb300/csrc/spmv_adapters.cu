// Low-rank adapters of many requests beside a shared projection
// (spmv_adapters_run): y_t = base_t + scale_s * B_s (A_s x_t), s the slot of
// token t.
//
// Two products of small inner size: h = A_s x_t is bound by reading x (and
// A_s, shared by the slot's tokens), y += B_s h by reading base and writing
// y. Both run on warp-level matrix instructions (16 x 8 x 16, fp32
// accumulation) whose operands go straight from global memory to registers:
// the order of the inner index is free as long as both operands agree on it,
// so lane t of a row takes 8 neighbouring elements (one 16-byte load) as its
// share of 32 and no shared-memory staging or transposition is needed. At
// ranks of 16 to 64 that is 8 to 30 operations per byte of x and y, far below
// what would fill the tensor cores, so the instruction's rate does not matter.
//
// h is kept in fp32 and enters the second product as a sum of 16-bit terms:
// two fp16 terms after scaling each token's h by a power of two (22 bits
// below its largest element), or three bf16 terms (24 bits).
#include <cooperative_groups.h>

#include <climits>
#include <type_traits>

#include "spmv_device.cuh"
#include "spmv_types.cuh"

namespace spmv {
namespace {

namespace cg = cooperative_groups;

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
  bool vec_in;   // rows of x and A: 16-byte aligned, n_in a multiple of 8
  bool vec_b;    // rows of B: the same, with rank
  bool vec_y;    // rows of base and y: 4 elements aligned, n_out a multiple of 4
  // grouped tokens (workspace)
  int4* tiles;       // {slot or -1, first sorted position, tokens, unused}
  int32_t* n_tiles;
  int32_t* perm;     // token at each sorted position
  float* parts;      // k_split x n_tokens (sorted) x rank partial sums of h
  int max_tiles, k_split, o_split;
};

template <typename T>
struct Terms;  // 16-bit terms of an fp32 h
template <>
struct Terms<__half> { static constexpr int n = 2; };
template <>
struct Terms<__nv_bfloat16> { static constexpr int n = 3; };

__device__ __forceinline__ void mma(const __half*, float (&c)[4], uint32_t a0, uint32_t a1,
                                    uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(const __nv_bfloat16*, float (&c)[4], uint32_t a0, uint32_t a1,
                                    uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// c += (rows lo: g, hi: g + 8 of 16) x (columns), over 32 inner elements.
template <typename T>
__device__ __forceinline__ void mma32(float (&c)[4], const uint4& lo, const uint4& hi,
                                      const uint4& v) {
  mma(static_cast<const T*>(nullptr), c, lo.x, hi.x, lo.y, hi.y, v.x, v.y);
  mma(static_cast<const T*>(nullptr), c, lo.z, hi.z, lo.w, hi.w, v.z, v.w);
}

// 8 elements at p of which `left` exist (the others are zero); vec: p is
// 16-byte aligned and all 8 or none exist.
template <typename T>
__device__ __forceinline__ uint4 load8(const T* p, int left, bool vec) {
  if (vec) return left > 0 ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
  const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
  uint32_t e[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) e[k] = k < left ? __ldg(q + k) : 0u;
  return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}

// The first `left` of 8 elements, zeros in place of the others.
__device__ __forceinline__ uint4 keep8(uint4 v, int left) {
  const auto word = [&](uint32_t w, int i) {
    return left >= 2 * i + 2 ? w : left == 2 * i + 1 ? w & 0xffffu : 0u;
  };
  return make_uint4(word(v.x, 0), word(v.y, 1), word(v.z, 2), word(v.w, 3));
}

__device__ __forceinline__ int rank_of(const AdapterArgs& p, int slot) {
  return p.ranks ? min(max(p.ranks[slot], 0), p.rank) : p.rank;
}

// acc[mt][nt] += rows j0 + 16 mt .. of A times tokens 8 nt .. over the inner
// range [k0, k1), in steps of 32 that start at k0 + 32 * first and are
// 32 * step apart. Rows past the rank repeat its last row (their h is not
// used); x[nt] is the row of this lane's token, any row where there is none.
template <typename T, int MT, int NT>
__device__ __forceinline__ void shrink(const AdapterArgs& p, const T* a, int rank, int j0,
                                       const T* const (&x)[NT], int k0, int k1,
                                       float (&acc)[MT][NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const T* rows[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      rows[m][h] = a + (int64_t)min(j0 + 16 * m + 8 * h + g, rank - 1) * p.n_in + 8 * t;
  const int whole = p.vec_in ? min(k1, p.n_in / 32 * 32) : k0;
  int k = k0;
#pragma unroll 2
  for (; k < whole; k += 32) {
    uint4 v[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n)
      v[n] = __ldg(reinterpret_cast<const uint4*>(x[n] + k + 8 * t));
    uint4 w[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) w[m][h] = __ldg(reinterpret_cast<const uint4*>(rows[m][h] + k));
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) mma32<T>(acc[m][n], w[m][0], w[m][1], v[n]);
  }
  for (; k < k1; k += 32) {  // the last, partial step; all steps of unaligned rows
    const int left = p.n_in - k - 8 * t;
    uint4 v[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) v[n] = load8(x[n] + k + 8 * t, left, p.vec_in);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint4 lo = load8(rows[m][0] + k, left, p.vec_in);
      const uint4 hi = load8(rows[m][1] + k, left, p.vec_in);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma32<T>(acc[m][n], lo, hi, v[n]);
    }
  }
}

// Write a token's h as 16-bit terms, by one warp: element j of lane j % 32 in
// v[j / 32] (0 past the rank). Returns the power of two that undoes the
// scaling. `pitch`: elements between terms.
template <typename T>
__device__ __forceinline__ float split_terms(const float (&v)[SPMV_ADAPTER_MAX_RANK / 32], int nk,
                                             T* out, int pitch) {
  const int lane = threadIdx.x & 31;
  float up = 1.f, down = 1.f;
  if constexpr (std::is_same<T, __half>::value) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < SPMV_ADAPTER_MAX_RANK / 32; ++i)
      if (i < nk) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // the largest element to [2^13, 2^14); 0, infinities and fp32's very
    // smallest stay as they are
    const int e = (int)((__float_as_uint(m) >> 23) & 255) - 127;
    if (e >= -113 && e < 128) {
      up = __uint_as_float((uint32_t)(13 - e + 127) << 23);
      down = __uint_as_float((uint32_t)(e - 13 + 127) << 23);
    }
  }
#pragma unroll
  for (int i = 0; i < SPMV_ADAPTER_MAX_RANK / 32; ++i) {
    if (i >= nk) break;
    float rest = v[i] * up;
#pragma unroll
    for (int k = 0; k < Terms<T>::n; ++k) {
      const T term = from_f32<T>(rest);
      out[k * pitch + i * 32 + lane] = term;
      // an infinite or NaN term is passed on once
      rest = isfinite(to_f32(term)) ? rest - to_f32(term) : 0.f;
    }
  }
  return down;
}

// acc[m][n]: columns o + 4 g + 2 m (and + 1) of y, tokens 8 n + 2 t (and + 1):
// lane rows of the two 16-row tiles are laid out so that a lane ends with 4
// neighbouring columns of each of its tokens. h: terms of 8 NT tokens,
// `pitch_t` elements per token and `pitch_k` per term.
template <typename T, int NT>
__device__ __forceinline__ void expand(const AdapterArgs& p, const T* b, int rank, int nk, int o,
                                       const T* h, int pitch_t, int pitch_k,
                                       float (&acc)[2][NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const T* rows[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    rows[i] = b + (int64_t)min(o + 4 * g + i, p.n_out - 1) * p.rank + 8 * t;
#pragma unroll 2
  for (int k = 0; k < nk; ++k) {
    uint4 w[4];
    const int left = rank - 32 * k - 8 * t;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = load8(rows[i] + 32 * k, left, p.vec_b);
    if (left < 8) {  // columns past the slot's rank
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = keep8(w[i], left);
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const T* hp = h + (8 * n + g) * pitch_t + 32 * k + 8 * t;
#pragma unroll
      for (int q = 0; q < Terms<T>::n; ++q) {
        const uint4 v = *reinterpret_cast<const uint4*>(hp + q * pitch_k);
        mma32<T>(acc[0][n], w[0], w[1], v);
        mma32<T>(acc[1][n], w[2], w[3], v);
      }
    }
  }
}

// 4 neighbouring columns of y, `left` of which exist.
template <typename YT>
__device__ __forceinline__ float4 load_y(const YT* p, int left, bool vec) {
  if (vec) {
    if (left <= 0) return make_float4(0, 0, 0, 0);
    const Pack<YT, 4> r = load_pack<YT, 4>(p, true);
    return make_float4(to_f32(r.v[0]), to_f32(r.v[1]), to_f32(r.v[2]), to_f32(r.v[3]));
  }
  return make_float4(left > 0 ? to_f32(p[0]) : 0.f, left > 1 ? to_f32(p[1]) : 0.f,
                     left > 2 ? to_f32(p[2]) : 0.f, left > 3 ? to_f32(p[3]) : 0.f);
}
template <typename YT>
__device__ __forceinline__ void store_y(YT* p, float4 v, int left, bool vec) {
  if (vec) {
    if (left <= 0) return;
    Pack<YT, 4> r;
    r.v[0] = from_f32<YT>(v.x);
    r.v[1] = from_f32<YT>(v.y);
    r.v[2] = from_f32<YT>(v.z);
    r.v[3] = from_f32<YT>(v.w);
    store_pack<YT, 4>(p, r);
    return;
  }
  if (left > 0) p[0] = from_f32<YT>(v.x);
  if (left > 1) p[1] = from_f32<YT>(v.y);
  if (left > 2) p[2] = from_f32<YT>(v.z);
  if (left > 3) p[3] = from_f32<YT>(v.w);
}

// y = base (or 0) for columns [o0, o1) of a token, by the whole CTA.
template <typename YT>
__device__ __forceinline__ void copy_base(const AdapterArgs& p, int token, int o0, int o1) {
  if (p.base == p.y) return;
  const YT* base = static_cast<const YT*>(p.base) + (p.base ? token * p.bs : 0);
  YT* y = static_cast<YT*>(p.y) + token * p.ys;
  for (int o = o0 + 4 * threadIdx.x; o < o1; o += 4 * blockDim.x)
    store_y(y + o, p.base ? load_y(base + o, o1 - o, p.vec_y) : make_float4(0, 0, 0, 0), o1 - o,
            p.vec_y);
}

// Add the product to base for one step of 32 columns x 8 NT tokens and store.
template <typename YT, int NT>
__device__ __forceinline__ void finish(const AdapterArgs& p, const int* s_token, int n_tokens,
                                       const float* s_down, float scale, int o,
                                       const float (&acc)[2][NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int c = o + 4 * g, left = p.n_out - c;
  float4 v[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 8 * n + 2 * t + e;
      v[n][e] = make_float4(0, 0, 0, 0);
      if (p.base && i < n_tokens)
        v[n][e] = load_y(static_cast<const YT*>(p.base) + s_token[i] * p.bs + c, left, p.vec_y);
    }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 8 * n + 2 * t + e;
      if (i >= n_tokens) continue;
      const float d = s_down[i];
      float4 r = v[n][e];
      r.x += scale * (acc[0][n][e] * d);
      r.y += scale * (acc[0][n][2 + e] * d);
      r.z += scale * (acc[1][n][e] * d);
      r.w += scale * (acc[1][n][2 + e] * d);
      store_y(static_cast<YT*>(p.y) + s_token[i] * p.ys + c, r, left, p.vec_y);
    }
}

constexpr int kMaxRank = SPMV_ADAPTER_MAX_RANK;
constexpr int kPitch = kMaxRank + 8;  // 16-bit elements per token: rows on other banks

// ------------------------------------------------------- few tokens (decode)
// A cluster of CTAs per token, of which the cluster of the first of every
// eight tokens of a slot works for all eight (a matrix instruction has eight
// columns) and the others leave at once. Each CTA takes a share of the inner
// range of A x; the shares meet in distributed shared memory; then each CTA
// takes a share of y's columns. One launch, no workspace; what B's share will
// need is asked from L2 at the start.
constexpr int kFewTokens = 256;
constexpr int kGroup = 8;

template <typename T, int MT>
__device__ __forceinline__ void few_shrink(const AdapterArgs& p, const T* a, int rank, int j0,
                                           const T* x, int k0, int k1, float* s_warp,
                                           float* s_part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // the warps' shares: neighbouring steps of 32
  const int steps = (k1 - k0 + 31) / 32, per = (steps + kWarps - 1) / kWarps;
  const int w0 = min(k0 + warp * per * 32, k1), w1 = min(w0 + per * 32, k1);
  float acc[MT][1][4] = {};
  const T* const xs[1] = {x};
  shrink<T, MT, 1>(p, a, rank, j0, xs, w0, w1, acc);
  // [warp][token][16 MT]
  float* mine = s_warp + warp * kGroup * 16 * MT;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      mine[(2 * t + (e & 1)) * 16 * MT + 16 * m + g + 8 * (e >> 1)] = acc[m][0][e];
  __syncthreads();
  for (int i = threadIdx.x; i < kGroup * 16 * MT; i += kThreads) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += s_warp[w * kGroup * 16 * MT + i];
    const int token = i / (16 * MT), j = j0 + i % (16 * MT);
    if (j < kMaxRank) s_part[token * kMaxRank + j] = v;
  }
  __syncthreads();
}

template <typename T, typename YT>
__global__ void __launch_bounds__(kThreads) adapters_few(AdapterArgs p) {
  __shared__ uint32_t s_same[kFewTokens / 32];
  __shared__ int s_token[kGroup];
  __shared__ float s_down[kGroup];
  __shared__ float s_warp[kWarps * kGroup * 64];
  __shared__ float s_part[kGroup * kMaxRank];
  __shared__ __align__(16) T s_h[Terms<T>::n * kGroup * kPitch];
  cg::cluster_group cluster = cg::this_cluster();
  const int ctas = cluster.num_blocks(), cta = cluster.block_rank();
  const int token = blockIdx.x / ctas, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int slot = p.ids[token];
  const int o_per = (p.n_out + 32 * ctas - 1) / (32 * ctas) * 32;
  const int o0 = min(cta * o_per, p.n_out), o1 = min(o0 + o_per, p.n_out);
  const int rank = slot >= 0 && slot < p.n_slots ? rank_of(p, slot) : 0;
  if (rank == 0) {
    copy_base<YT>(p, token, o0, o1);
    return;
  }
  // tokens of the same slot
  for (int i = warp; i < (p.n_tokens + 31) / 32; i += kWarps) {
    const int at = i * 32 + lane;
    const uint32_t m = __ballot_sync(0xffffffffu, at < p.n_tokens && p.ids[at] == slot);
    if (lane == 0) s_same[i] = m;
  }
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < (p.n_tokens + 31) / 32; ++i) {
    const uint32_t m = s_same[i];
    all += __popc(m);
    before += i < token / 32 ? __popc(m)
              : i == token / 32 ? __popc(m & ((1u << (token % 32)) - 1)) : 0;
  }
  if (before % kGroup) return;  // (the whole cluster)
  const int n_tokens = min(all - before, kGroup);
  if ((int)threadIdx.x < n_tokens) {
    int skip = before + threadIdx.x, i = 0;
    while (skip >= __popc(s_same[i])) skip -= __popc(s_same[i++]);
    uint32_t m = s_same[i];
    while (skip--) m &= m - 1;
    s_token[threadIdx.x] = i * 32 + __ffs(m) - 1;
  }
  __syncthreads();

  const T* b = static_cast<const T*>(p.b) + (int64_t)slot * p.n_out * p.rank;
  if (o1 > o0) {
    const char* from = reinterpret_cast<const char*>(b + (int64_t)o0 * p.rank);
    const int64_t bytes = (int64_t)(o1 - o0) * p.rank * (int)sizeof(T);
    for (int64_t i = 128ll * threadIdx.x; i < bytes; i += 128ll * kThreads)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(from + i));
  }
  const int k_per = (p.n_in + 32 * ctas - 1) / (32 * ctas) * 32;
  const int k0 = min(cta * k_per, p.n_in), k1 = min(k0 + k_per, p.n_in);
  const T* a = static_cast<const T*>(p.a) + (int64_t)slot * p.rank * p.n_in;
  const T* x = static_cast<const T*>(p.x) + s_token[min(lane >> 2, n_tokens - 1)] * p.xs;
  if (rank <= 16)
    few_shrink<T, 1>(p, a, rank, 0, x, k0, k1, s_warp, s_part);
  else if (rank <= 32)
    few_shrink<T, 2>(p, a, rank, 0, x, k0, k1, s_warp, s_part);
  else
    for (int j0 = 0; j0 < rank; j0 += 64)
      few_shrink<T, 4>(p, a, rank, j0, x, k0, k1, s_warp, s_part);
  cluster.sync();
  const int nk = (rank + 31) / 32;
  if (warp < n_tokens) {  // a warp per token: its h over the cluster's shares
    float v[kMaxRank / 32];
#pragma unroll
    for (int i = 0; i < kMaxRank / 32; ++i) {
      v[i] = 0.f;
      if (i < nk && i * 32 + lane < rank)
        for (int c = 0; c < ctas; ++c)
          v[i] += cluster.map_shared_rank(s_part, c)[warp * kMaxRank + i * 32 + lane];
    }
    const float down = split_terms<T>(v, nk, s_h + warp * kPitch, kGroup * kPitch);
    if (lane == 0) s_down[warp] = down;
  } else {  // columns of the matrix instruction that no token has
    for (int k = 0; k < Terms<T>::n; ++k)
      for (int j = lane; j < kPitch; j += 32)
        s_h[(k * kGroup + warp) * kPitch + j] = from_f32<T>(0.f);
  }
  __syncthreads();
  // the others may still read this CTA's share: its memory goes after them
  asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  const float scale = p.scales ? p.scales[slot] : 1.f;
  for (int o = o0 + 32 * warp; o < o1; o += 32 * kWarps) {
    float acc[2][1][4] = {};
    expand<T, 1>(p, b, rank, nk, o, s_h, kPitch, kGroup * kPitch, acc);
    finish<YT, 1>(p, s_token, n_tokens, s_down, scale, o, acc);
  }
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

// --------------------------------------------------- many tokens (prompts)
// Tokens are first sorted by slot and cut into tiles of one slot's tokens;
// then A x per tile and share of the inner range, and y per tile and share of
// the columns.
constexpr int kTile = 64;
constexpr int kSortThreads = 1024;

__global__ void __launch_bounds__(kSortThreads) adapters_sort(AdapterArgs p) {
  extern __shared__ int s_count[];  // per slot, the tokens without one last
  __shared__ int2 s_warp[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = p.n_slots + 1;
  for (int i = threadIdx.x; i < n; i += kSortThreads) s_count[i] = 0;
  __syncthreads();
  const auto slot_at = [&](int i) {
    const int s = p.ids[i];
    return s >= 0 && s < p.n_slots ? s : p.n_slots;
  };
  // one atomic for the lanes of a warp that share a slot
  const int rounds = (p.n_tokens + kSortThreads - 1) / kSortThreads;
  for (int q = 0; q < rounds; ++q) {
    const int i = q * kSortThreads + threadIdx.x;
    const int s = i < p.n_tokens ? slot_at(i) : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, s);
    if (s >= 0 && lane == __ffs(same) - 1) atomicAdd(&s_count[s], __popc(same));
  }
  __syncthreads();
  // running sums of tokens and of tiles, a run of slots per thread
  const int per = (n + kSortThreads - 1) / kSortThreads;
  const int lo = min((int)threadIdx.x * per, n), hi = min(lo + per, n);
  int2 v = make_int2(0, 0);
  for (int i = lo; i < hi; ++i) {
    v.x += s_count[i];
    v.y += (s_count[i] + kTile - 1) / kTile;
  }
  int2 sum = v;
  for (int o = 1; o < 32; o <<= 1) {
    const int a = __shfl_up_sync(0xffffffffu, sum.x, o), b = __shfl_up_sync(0xffffffffu, sum.y, o);
    if (lane >= o) sum.x += a, sum.y += b;
  }
  if (lane == 31) s_warp[warp] = sum;
  __syncthreads();
  int2 at = make_int2(sum.x - v.x, sum.y - v.y);
  for (int w = 0; w < warp; ++w) at.x += s_warp[w].x, at.y += s_warp[w].y;
  for (int i = lo; i < hi; ++i) {
    const int tokens = s_count[i];
    s_count[i] = at.x;
    for (int k = 0; k < tokens; k += kTile)
      p.tiles[at.y++] = make_int4(i < p.n_slots ? i : -1, at.x + k, min(kTile, tokens - k), 0);
    at.x += tokens;
  }
  if (threadIdx.x == kSortThreads - 1) *p.n_tiles = at.y;
  __syncthreads();
  for (int q = 0; q < rounds; ++q) {
    const int i = q * kSortThreads + threadIdx.x;
    const int s = i < p.n_tokens ? slot_at(i) : -1;
    const uint32_t same = __match_any_sync(0xffffffffu, s);
    const int first = __ffs(same) - 1;
    int base = 0;
    if (s >= 0 && lane == first) base = atomicAdd(&s_count[s], __popc(same));
    base = __shfl_sync(0xffffffffu, base, first);
    // the order of a slot's tokens does not change any token's result
    if (s >= 0) p.perm[base + __popc(same & ((1u << lane) - 1))] = i;
  }
}

// Warps of a CTA: two halves of the tile's tokens times four shares of the
// CTA's inner range.
template <typename T, int MT>
__device__ __forceinline__ void tile_shrink(const AdapterArgs& p, const T* a, int rank, int j0,
                                            const T* const (&x)[4], int n_tokens, int start,
                                            int split, int k0, int k1, float* s_sum) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int half = warp & 1, share = warp >> 1;
  const int steps = (k1 - k0 + 31) / 32, per = (steps + 3) / 4;
  const int w0 = min(k0 + share * per * 32, k1), w1 = min(w0 + per * 32, k1);
  float acc[MT][4][4] = {};
  if (half * 32 < n_tokens) shrink<T, MT, 4>(p, a, rank, j0, x, w0, w1, acc);
  // s_sum: [token][16 MT], added up share by share
  for (int s = 0; s < 4; ++s) {
    if (share == s) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float* at = s_sum + (32 * half + 8 * n + 2 * t + (e & 1)) * (16 * MT + 1) + 16 * m +
                        g + 8 * (e >> 1);
            *at = s ? *at + acc[m][n][e] : acc[m][n][e];
          }
    }
    __syncthreads();
  }
  const int width = min(16 * MT, rank - j0);
  for (int i = threadIdx.x; i < n_tokens * width; i += kThreads) {
    const int token = i / width, j = i % width;
    p.parts[((int64_t)split * p.n_tokens + start + token) * p.rank + j0 + j] =
        s_sum[token * (16 * MT + 1) + j];
  }
  __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) adapters_shrink(AdapterArgs p) {
  __shared__ float s_sum[kTile * 65];
  pdl_wait();
  const int split = blockIdx.x % p.k_split, i = blockIdx.x / p.k_split;
  if (i >= *p.n_tiles) return;
  const int4 tile = p.tiles[i];
  if (tile.x < 0) return;
  const int rank = rank_of(p, tile.x);
  if (rank == 0) return;
  const int k_per = (p.n_in + 32 * p.k_split - 1) / (32 * p.k_split) * 32;
  const int k0 = min(split * k_per, p.n_in), k1 = min(k0 + k_per, p.n_in);
  const T* a = static_cast<const T*>(p.a) + (int64_t)tile.x * p.rank * p.n_in;
  const int g = (threadIdx.x & 31) >> 2, half = (threadIdx.x >> 5) & 1;
  const T* x[4];
#pragma unroll
  for (int n = 0; n < 4; ++n)
    x[n] = static_cast<const T*>(p.x) +
           p.perm[tile.y + min(32 * half + 8 * n + g, tile.z - 1)] * p.xs;
  if (rank <= 16)
    tile_shrink<T, 1>(p, a, rank, 0, x, tile.z, tile.y, split, k0, k1, s_sum);
  else if (rank <= 32)
    tile_shrink<T, 2>(p, a, rank, 0, x, tile.z, tile.y, split, k0, k1, s_sum);
  else
    for (int j0 = 0; j0 < rank; j0 += 64)
      tile_shrink<T, 4>(p, a, rank, j0, x, tile.z, tile.y, split, k0, k1, s_sum);
  pdl_launch_dependents();
}

template <typename T, typename YT>
__global__ void __launch_bounds__(kThreads, 2) adapters_expand(AdapterArgs p) {
  extern __shared__ __align__(16) unsigned char s_dyn[];
  T* s_h = reinterpret_cast<T*>(s_dyn);  // [term][token][pitch]
  __shared__ int s_token[kTile];
  __shared__ float s_down[kTile];
  const int split = blockIdx.x % p.o_split, i = blockIdx.x / p.o_split;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  if (i >= *p.n_tiles) return;
  const int4 tile = p.tiles[i];
  const int o_per = (p.n_out + 32 * p.o_split - 1) / (32 * p.o_split) * 32;
  const int o0 = min(split * o_per, p.n_out), o1 = min(o0 + o_per, p.n_out);
  const int rank = tile.x < 0 ? 0 : rank_of(p, tile.x);
  if (rank == 0) {
    for (int k = 0; k < tile.z; ++k) copy_base<YT>(p, p.perm[tile.y + k], o0, o1);
    return;
  }
  const int nk = (rank + 31) / 32, pitch = 32 * ((p.rank + 31) / 32) + 8;
  if (threadIdx.x < kTile)
    s_token[threadIdx.x] = p.perm[tile.y + min((int)threadIdx.x, tile.z - 1)];
  for (int k = warp; k < kTile; k += kWarps) {
    float v[kMaxRank / 32];
#pragma unroll
    for (int q = 0; q < kMaxRank / 32; ++q) {
      v[q] = 0.f;
      if (q < nk && q * 32 + lane < rank && k < tile.z)
        for (int s = 0; s < p.k_split; ++s)
          v[q] += p.parts[((int64_t)s * p.n_tokens + tile.y + k) * p.rank + q * 32 + lane];
    }
    const float down = split_terms<T>(v, nk, s_h + k * pitch, kTile * pitch);
    if (lane == 0) s_down[k] = down;
  }
  __syncthreads();
  const T* b = static_cast<const T*>(p.b) + (int64_t)tile.x * p.n_out * p.rank;
  const float scale = p.scales ? p.scales[tile.x] : 1.f;
  const int half = warp & 1;
  if (32 * half >= tile.z) return;
  for (int o = o0 + 32 * (warp >> 1); o < o1; o += 32 * kWarps / 2) {
    float acc[2][4][4] = {};
    expand<T, 4>(p, b, rank, nk, o, s_h + 32 * half * pitch, pitch, kTile * pitch, acc);
    finish<YT, 4>(p, s_token + 32 * half, tile.z - 32 * half, s_down + 32 * half, scale, o, acc);
  }
}

constexpr int kMaxTokens = 1 << 27, kMaxWidth = 1 << 30;  // (32-bit grids and columns)

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Workspace of the sorted path: tile count, tiles, sorted tokens, partial h.
struct Workspace {
  int64_t tiles, perm, parts, bytes;
  int max_tiles, k_split;
};

Workspace workspace_of(int n_tokens, int n_slots, int rank) {
  Workspace w{};
  if (n_tokens <= kFewTokens || n_slots == 0 || rank == 0) return w;
  w.max_tiles = n_tokens / kTile + (n_slots + 1 < n_tokens ? n_slots + 1 : n_tokens);
  const int tiles = (n_tokens + kTile - 1) / kTile;
  w.k_split = tiles >= 304 ? 1 : (304 + tiles - 1) / tiles;
  if (w.k_split > 8) w.k_split = 8;
  w.tiles = 16;
  w.perm = round_up(w.tiles + 16ll * w.max_tiles, 128);
  w.parts = round_up(w.perm + 4ll * n_tokens, 128);
  w.bytes = w.parts + 4ll * w.k_split * n_tokens * rank;
  return w;
}

template <typename T, typename YT>
spmv_status run_few(AdapterArgs& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  const int ctas = 8;
  cfg.gridDim = dim3((unsigned)(p.n_tokens * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {&p};
  return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(&adapters_few<T, YT>), args) ==
                 cudaSuccess
             ? SPMV_OK
             : SPMV_ERR_CUDA;
}

template <typename T, typename YT>
spmv_status run_many(AdapterArgs& p, cudaStream_t st) {
  const int tiles = (p.n_tokens + kTile - 1) / kTile;
  const int most = (p.n_out + 127) / 128;  // a CTA step is 128 columns
  p.o_split = (912 + tiles - 1) / tiles;
  p.o_split = p.o_split < 1 ? 1 : p.o_split > most ? most : p.o_split;
  const size_t sort_smem = (size_t)(p.n_slots + 1) * 4;
  const size_t expand_smem =
      (size_t)Terms<T>::n * kTile * (32 * ((p.rank + 31) / 32) + 8) * sizeof(T);
  if ((int64_t)p.max_tiles * p.o_split > INT_MAX) return SPMV_ERR_TOO_LARGE;
  if ((sort_smem > 40 * 1024 &&
       cudaFuncSetAttribute(reinterpret_cast<const void*>(&adapters_sort),
                            cudaFuncAttributeMaxDynamicSharedMemorySize,
                            (int)sort_smem) != cudaSuccess) ||
      (expand_smem > 40 * 1024 &&
       cudaFuncSetAttribute(reinterpret_cast<const void*>(&adapters_expand<T, YT>),
                            cudaFuncAttributeMaxDynamicSharedMemorySize,
                            (int)expand_smem) != cudaSuccess))
    return SPMV_ERR_CUDA;
  adapters_sort<<<1, kSortThreads, sort_smem, st>>>(p);
  if (cudaGetLastError() != cudaSuccess) return SPMV_ERR_CUDA;
  void* args[] = {&p};
  if (launch_pdl(reinterpret_cast<const void*>(&adapters_shrink<T>), p.max_tiles * p.k_split,
                 kThreads, 0, st, args) != 0 ||
      launch_pdl(reinterpret_cast<const void*>(&adapters_expand<T, YT>), p.max_tiles * p.o_split,
                 kThreads, expand_smem, st, args) != 0)
    return SPMV_ERR_CUDA;
  return SPMV_OK;
}

template <typename T, typename YT>
spmv_status run(AdapterArgs& p, cudaStream_t st) {
  return p.n_tokens <= kFewTokens || !p.parts ? run_few<T, YT>(p, st) : run_many<T, YT>(p, st);
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" int64_t spmv_adapters_workspace(int32_t n_tokens, int32_t n_slots, int32_t rank) {
  if (n_tokens < 0 || n_slots < 0 || rank < 0 || rank > SPMV_ADAPTER_MAX_RANK ||
      n_slots > SPMV_ADAPTER_MAX_SLOTS || n_tokens > kMaxTokens)
    return 0;
  return workspace_of(n_tokens, n_slots, rank).bytes;
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
  if (rank > SPMV_ADAPTER_MAX_RANK || n_slots > SPMV_ADAPTER_MAX_SLOTS ||
      n_tokens > kMaxTokens || n_in > kMaxWidth || n_out > kMaxWidth)
    return SPMV_ERR_TOO_LARGE;
  const int64_t ysz = op_dtype_size(y_dtype);
  const bool weights = n_slots > 0 && rank > 0;
  if (!matrix_ok(x, n_tokens, n_in, x_stride, 2, false) ||
      (base && !matrix_ok(base, n_tokens, n_out, base_stride, ysz, false)) ||
      !matrix_ok(y, n_tokens, n_out, y_stride, ysz, true) ||
      (weights && ((n_in > 0 && !a) || (n_out > 0 && !b))) || !aligned_to(a, 2) ||
      !aligned_to(b, 2) || (n_tokens > 0 && !slot_ids) || !aligned_to(slot_ids, 4) ||
      !aligned_to(ranks, 4) || !aligned_to(scales, 4) || !aligned_to(workspace, 16))
    return SPMV_ERR_INVALID_ARG;
  const Workspace w = workspace_of(n_tokens, n_slots, rank);
  if (w.bytes > 0 && (!workspace || workspace_bytes < w.bytes)) return SPMV_ERR_INVALID_ARG;
  if (n_tokens == 0 || n_out == 0) return SPMV_OK;
  const bool in_place = base == y && (base_stride == y_stride || n_tokens == 1);
  if ((!in_place && spans_overlap(base, n_tokens, n_out, base_stride, ysz, y, n_tokens, n_out,
                                  y_stride, ysz)) ||
      spans_overlap(x, n_tokens, n_in, x_stride, 2, y, n_tokens, n_out, y_stride, ysz))
    return SPMV_ERR_INVALID_ARG;
  AdapterArgs p{};
  p.n_tokens = n_tokens, p.n_in = n_in, p.n_out = n_out;
  p.n_slots = weights && n_in > 0 ? n_slots : 0;  // (nothing to add: y = base)
  p.rank = rank;
  p.x = x, p.xs = x_stride, p.a = a, p.b = b, p.ids = slot_ids, p.ranks = ranks, p.scales = scales;
  p.base = base, p.bs = base_stride, p.y = y, p.ys = y_stride;
  p.vec_in = n_in % 8 == 0 && rows_aligned(x, n_tokens, x_stride, 2, 8) && aligned_to(a, 16);
  p.vec_b = rank % 8 == 0 && aligned_to(b, 16);
  p.vec_y = n_out % 4 == 0 && rows_aligned(y, n_tokens, y_stride, ysz, 4) &&
            (!base || rows_aligned(base, n_tokens, base_stride, ysz, 4));
  if (w.bytes > 0) {
    char* at = static_cast<char*>(workspace);
    p.n_tiles = reinterpret_cast<int32_t*>(at);
    p.tiles = reinterpret_cast<int4*>(at + w.tiles);
    p.perm = reinterpret_cast<int32_t*>(at + w.perm);
    p.parts = reinterpret_cast<float*>(at + w.parts);
    p.max_tiles = w.max_tiles, p.k_split = w.k_split;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SPMV_F16)
    return y_dtype == SPMV_F32 ? run<__half, float>(p, st) : run<__half, __half>(p, st);
  return y_dtype == SPMV_F32 ? run<__nv_bfloat16, float>(p, st)
                             : run<__nv_bfloat16, __nv_bfloat16>(p, st);
}
