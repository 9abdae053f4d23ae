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
// Measured at 12288 x 12288, fp16 x, fp32 base and y, in us and as a share of
// the 6.79 TB/s of a plain copy: 4096 tokens of 8 adapters at rank 32 117
// (0.65; the second product 74, at 0.81; the first 32, whose eight warps per SM
// wait for loads to registers; the sort 6), at rank 64 154 (0.51), 1024 tokens
// at rank 16 46 (0.42); 48 tokens of 32 adapters at rank 64 34 (0.37); one
// token at rank 16 10. Few tokens are bound by latency: two products one after
// the other, two trips to memory and a cluster's barrier between them.
//
// h is kept in fp32 and enters the second product as a sum of 16-bit terms:
// three bf16 terms (24 bits of each element), or two fp16 terms (22 bits, down
// to 2^-38 of the token's largest element) after scaling the token's h by a
// power of two. A third fp16 term would be half as many instructions again,
// for an error that the products' own fp32 sums exceed.
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
  int vec_in;    // rows of x and A, and n_in: 0 any, 1 whole 16 bytes, 2 whole 32 bytes
  int vec_b;     // rows of B, and rank: 0 any, 1 whole 16 bytes, 8 or 4: whole 8 or 4 bytes
  bool vec_y;    // rows of base and y: 4 elements aligned, n_out a multiple of 4
  // grouped tokens (workspace)
  int4* tiles;       // {slot or -1, first sorted position, tokens, unused}
  int32_t* n_tiles;
  int32_t* perm;     // token at each sorted position
  void* terms;       // 16-bit terms of h: [sorted position][term][term_pitch]
  float* downs;      // what undoes their scaling, per sorted position
  int term_pitch, max_tiles, k_split;
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

// 8 elements at p of which `left` exist (the others are zero), in the largest
// loads that `vec` allows: 1: 16 bytes, 8 or 4: that many, 0: single elements
// (rows are a whole number of such loads).
template <typename T>
__device__ __forceinline__ uint4 load8(const T* p, int left, int vec) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (vec == 1) {
    if (left > 0) v = __ldg(reinterpret_cast<const uint4*>(p));
  } else if (vec == 8) {
    const uint2* q = reinterpret_cast<const uint2*>(p);
    uint2 lo = make_uint2(0, 0), hi = lo;
    if (left > 0) lo = __ldg(q);
    if (left > 4) hi = __ldg(q + 1);
    v = make_uint4(lo.x, lo.y, hi.x, hi.y);
  } else if (vec == 4) {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
    if (left > 0) v.x = __ldg(q);
    if (left > 2) v.y = __ldg(q + 1);
    if (left > 4) v.z = __ldg(q + 2);
    if (left > 6) v.w = __ldg(q + 3);
  } else {
    const unsigned short* q = reinterpret_cast<const unsigned short*>(p);
    uint32_t e[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      e[k] = 0;
      if (k < left) e[k] = __ldg(q + k);
    }
    v = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
  }
  return v;
}

// 8 elements at any p (2-byte aligned) of which the 7 before and the 16 from p
// on exist too: the two 16-byte granules around them, shifted into place.
// (Against 8 loads of an element: a third of the L1 accesses.)
template <typename T>
__device__ __forceinline__ uint4 load8_shifted(const T* p) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const uint4* q = reinterpret_cast<const uint4*>(at & ~uintptr_t(15));
  const uint4 a = __ldg(q), b = __ldg(q + 1);
  const bool by2 = at & 8, by1 = at & 4;
  const uint32_t half = 8 * (uint32_t)(at & 2);
  // words from the one that holds p's element on
  const uint32_t u0 = by2 ? a.z : a.x, u1 = by2 ? a.w : a.y, u2 = by2 ? b.x : a.z,
                 u3 = by2 ? b.y : a.w, u4 = by2 ? b.z : b.x, u5 = by2 ? b.w : b.y;
  const uint32_t v0 = by1 ? u1 : u0, v1 = by1 ? u2 : u1, v2 = by1 ? u3 : u2, v3 = by1 ? u4 : u3,
                 v4 = by1 ? u5 : u4;
  return make_uint4(__funnelshift_r(v0, v1, half), __funnelshift_r(v1, v2, half),
                    __funnelshift_r(v2, v3, half), __funnelshift_r(v3, v4, half));
}

// 16 elements (32 bytes, aligned to it) in one load: a quarter-warp then
// covers two whole 128-byte lines.
struct Vec16 {
  uint32_t w[8];
};
__device__ __forceinline__ Vec16 load16(const void* p) {
  Vec16 r;
  asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]),
                 "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
               : "l"(p));
  return r;
}
// c += rows x columns over 64 inner elements.
template <typename T>
__device__ __forceinline__ void mma64(float (&c)[4], const Vec16& lo, const Vec16& hi,
                                      const Vec16& v) {
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    mma(static_cast<const T*>(nullptr), c, lo.w[i], hi.w[i], lo.w[i + 1], hi.w[i + 1], v.w[i],
        v.w[i + 1]);
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
// range [k0, k1), k0 a multiple of 64. Rows past the rank repeat its last row
// (their h is not used); x[nt] is the row of this lane's token, any row where
// there is none. ANY: rows of any alignment. MOST: the largest NT that the
// caller uses for these rows. The steps' length is chosen by it and not by NT,
// so that a token's sums are added in the same order in every tile.
template <typename T, int MT, int NT, int MOST, bool ANY>
__device__ __forceinline__ void shrink(const AdapterArgs& p, const T* a, int rank, int j0,
                                       const T* const (&x)[NT], int k0, int k1,
                                       float (&acc)[MT][NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const T* rows[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      rows[m][h] = a + (int64_t)min(j0 + 16 * m + 8 * h + g, rank - 1) * p.n_in;
  int k = k0;
  if constexpr (!ANY && MT * MOST <= 16) {  // (more would not fit the registers)
    const int whole = p.vec_in == 2 ? k0 + max(min(k1, p.n_in) - k0, 0) / 64 * 64 : k0;
    for (; k < whole; k += 64) {
      Vec16 v[NT], w[MT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) v[n] = load16(x[n] + k + 16 * t);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) w[m][h] = load16(rows[m][h] + k + 16 * t);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) mma64<T>(acc[m][n], w[m][0], w[m][1], v[n]);
    }
  }
  if constexpr (!ANY) {
    const int whole = k0 + max(min(k1, p.n_in) - k0, 0) / 32 * 32;
#pragma unroll 2
    for (; k < whole; k += 32) {
      uint4 v[NT], w[MT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) v[n] = __ldg(reinterpret_cast<const uint4*>(x[n] + k + 8 * t));
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[m][h] = __ldg(reinterpret_cast<const uint4*>(rows[m][h] + k + 8 * t));
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) mma32<T>(acc[m][n], w[m][0], w[m][1], v[n]);
    }
  }
  const auto single = [&] {
    const int left = p.n_in - k - 8 * t;
    uint4 v[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) v[n] = load8(x[n] + k + 8 * t, left, ANY ? 0 : 1);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const uint4 lo = load8(rows[m][0] + k + 8 * t, left, ANY ? 0 : 1);
      const uint4 hi = load8(rows[m][1] + k + 8 * t, left, ANY ? 0 : 1);
#pragma unroll
      for (int n = 0; n < NT; ++n) mma32<T>(acc[m][n], lo, hi, v[n]);
    }
  };
  if constexpr (ANY) {  // all but the first and last steps of a row
    if (k == 0 && k < k1) {
      single();
      k += 32;
    }
    for (; k < k1 && k + 40 <= p.n_in; k += 32) {
      uint4 v[NT], w[MT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) v[n] = load8_shifted(x[n] + k + 8 * t);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) w[m][h] = load8_shifted(rows[m][h] + k + 8 * t);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) mma32<T>(acc[m][n], w[m][0], w[m][1], v[n]);
    }
  }
  for (; k < k1; k += 32) single();
}

// Share i of n of the inner range, in whole steps of 64.
__device__ __forceinline__ int2 inner_share(int k0, int k1, int i, int n) {
  const int per = ((k1 - k0 + 63) / 64 + n - 1) / n * 64;
  const int lo = min(k0 + i * per, k1);
  return make_int2(lo, min(lo + per, k1));
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
      if (i < nk && isfinite(v[i])) m = fmaxf(m, fabsf(v[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // the largest finite element to [2^13, 2^14) (beside an infinite one they
    // must not become infinite themselves); 0 and fp32's very smallest stay as
    // they are
    const int e = (int)((__float_as_uint(m) >> 23) & 255) - 127;
    if (e >= -113) {
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

// 32 columns of B's rows o + 4 g + i, from column 32 k (zeros past the rank).
// Lane rows of the two 16-row tiles of a step are laid out so that a lane ends
// with 4 neighbouring columns of each of its tokens.
template <typename T>
__device__ __forceinline__ void load_b(const AdapterArgs& p, const T* b, int rank, int k, int o,
                                       uint4 (&w)[4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int left = rank - 32 * k - 8 * t;
  const T* at = b + 32 * k + 8 * t;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = load8(at + (int64_t)min(o + 4 * g + i, p.n_out - 1) * p.rank, left, p.vec_b);
  if (left < 8) {  // columns past the slot's rank
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = keep8(w[i], left);
  }
}

// acc[m][n][e + 2 i]: column o + 4 g + 2 m + i of y, token 8 n + 2 t + e, over
// the 32 inner elements of w. h: terms of 8 NT tokens at inner element 32 k,
// `pitch_t` elements per token and `pitch_k` per term.
template <typename T, int NT>
__device__ __forceinline__ void expand(const uint4 (&w)[4], const T* h, int pitch_t, int pitch_k,
                                       float (&acc)[2][NT][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int q = 0; q < Terms<T>::n; ++q) {
      const uint4 v =
          *reinterpret_cast<const uint4*>(h + (8 * n + g) * pitch_t + q * pitch_k + 8 * t);
      mma32<T>(acc[0][n], w[0], w[1], v);
      mma32<T>(acc[1][n], w[2], w[3], v);
    }
}

// 4 neighbouring columns of y, `left` of which exist (the others are zero).
template <typename YT>
__device__ __forceinline__ Pack<YT, 4> load_y(const YT* p, int left, bool vec) {
  if (vec && left > 0) return load_pack<YT, 4>(p, true);
  Pack<YT, 4> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.v[i] = !vec && i < left ? p[i] : from_f32<YT>(0.f);
  return r;
}
template <typename YT>
__device__ __forceinline__ void store_y(YT* p, const Pack<YT, 4>& r, int left, bool vec) {
  if (vec) {
    if (left > 0) store_pack<YT, 4>(p, r);
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) p[i] = r.v[i];
}

// y = base (or 0) for columns [o0, o1) of a token, by the whole CTA.
template <typename YT>
__device__ __forceinline__ void copy_base(const AdapterArgs& p, int token, int o0, int o1) {
  if (p.base == p.y) return;
  const YT* base = static_cast<const YT*>(p.base) + (p.base ? token * p.bs : 0);
  YT* y = static_cast<YT*>(p.y) + token * p.ys;
  for (int o = o0 + 4 * threadIdx.x; o < o1; o += 4 * blockDim.x)
    store_y(y + o, load_y(base + o, p.base ? o1 - o : 0, p.vec_y), o1 - o, p.vec_y);
}

// base and y are read and written by lanes in another order than the matrix
// instruction leaves them (lane 4 g + t -> 8 t + g): eight neighbouring lanes
// then cover one 128-byte line of one token, not 32 bytes of each of four
// (measured: 14 L1 wavefronts per 512-byte request before).
// The base of one step: columns o + 4 g .. of tokens 8 n + 2 t + e.
template <typename YT, int NT>
__device__ __forceinline__ void load_base(const AdapterArgs& p, const int* s_token, int n_tokens,
                                          int o, Pack<YT, 4> (&v)[NT][2]) {
  const int lane = threadIdx.x & 31, g = lane & 7, t = lane >> 3, c = o + 4 * g;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int i = 8 * n + 2 * t + e;
      const bool on = p.base && i < n_tokens;
      v[n][e] = load_y(static_cast<const YT*>(p.base) + (on ? s_token[i] * p.bs + c : 0),
                       on ? p.n_out - c : 0, p.vec_y);
    }
}

// Add the product to the base and store (whole warps).
template <typename YT, int NT>
__device__ __forceinline__ void finish(const AdapterArgs& p, const int* s_token, int n_tokens,
                                       const float* s_down, float scale, int o,
                                       const Pack<YT, 4> (&v)[NT][2],
                                       const float (&acc)[2][NT][4]) {
  const int lane = threadIdx.x & 31, g = lane & 7, t = lane >> 3, c = o + 4 * g;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float m[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        m[k] = __shfl_sync(0xffffffffu, acc[k >> 1][n][e + 2 * (k & 1)], 4 * g + t);
      const int i = 8 * n + 2 * t + e;
      if (i >= n_tokens) continue;
      const float d = s_down[i];
      Pack<YT, 4> r;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        r.v[k] = from_f32<YT>(to_f32(v[n][e].v[k]) + scale * (m[k] * d));
      store_y(static_cast<YT*>(p.y) + s_token[i] * p.ys + c, r, p.n_out - c, p.vec_y);
    }
}

constexpr int kMaxRank = SPMV_ADAPTER_MAX_RANK;
constexpr int kPitch = kMaxRank + 8;  // 16-bit elements per token: rows on other banks

// ------------------------------------------------------- few tokens (decode)
// Clusters of CTAs take groups of up to eight tokens of one slot (a matrix
// instruction has eight columns) in turn; which tokens form the groups every
// CTA finds for itself. Each CTA takes a share of the inner
// range of A x; the shares meet in distributed shared memory; then each CTA
// takes a share of y's columns. One launch, no workspace. What the second
// product needs does not depend on the first: B's share is asked from L2, and
// the first step's B and base are loaded, before the shares meet.
//
// A thread of the smallest CTA looks at each token, hence 256 tokens at most.
// (256 tokens of 64 adapters at rank 16, 12288 x 12288: 43 us; sorted, 62.)
constexpr int kFewTokens = 256;
constexpr int kGroup = 8;

// Shared memory of a CTA: the warps' sums of A x, later the 16-bit terms.
template <typename T, int WARPS>
union FewShared {
  float warps[WARPS * kGroup * 64];
  T h[Terms<T>::n * kGroup * kPitch];
};

template <typename T, int MT, int WARPS, bool ANY>
__device__ __forceinline__ void few_shrink(const AdapterArgs& p, const T* a, int rank, int j0,
                                           const T* x, int k0, int k1, float* s_warp,
                                           float* s_part) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int2 mine_k = inner_share(k0, k1, warp, WARPS);
  float acc[MT][1][4] = {};
  const T* const xs[1] = {x};
  shrink<T, MT, 1, 1, ANY>(p, a, rank, j0, xs, mine_k.x, mine_k.y, acc);
  // [warp][token][16 MT]
  float* mine = s_warp + warp * kGroup * 16 * MT;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      mine[(2 * t + (e & 1)) * 16 * MT + 16 * m + g + 8 * (e >> 1)] = acc[m][0][e];
  __syncthreads();
  for (int i = threadIdx.x; i < kGroup * 16 * MT; i += 32 * WARPS) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) v += s_warp[w * kGroup * 16 * MT + i];
    const int token = i / (16 * MT), j = j0 + i % (16 * MT);
    if (j < kMaxRank) s_part[token * kMaxRank + j] = v;
  }
  __syncthreads();
}

// The call's groups: first token of each, and how many tokens of its slot
// stand before it. Returns their number. (Whole CTA.)
template <int WARPS>
__device__ __forceinline__ int few_groups(const AdapterArgs& p, int* s_ids, int2* s_group) {
  __shared__ uint32_t s_first[kFewTokens / 32];
  static_assert(kFewTokens <= 32 * WARPS, "a thread per token");
  const int i = threadIdx.x, warp = i >> 5, lane = i & 31;
  if (i < kFewTokens) {
    const int id = i < p.n_tokens ? p.ids[i] : 0;
    s_ids[i] = id >= 0 && id < p.n_slots ? id : -1;
  }
  __syncthreads();
  int before = 0;
  bool first = false;
  if (i < p.n_tokens) {
    const int id = s_ids[i];
    for (int j = 0; j < i; j += 4) {
      const int4 v = *reinterpret_cast<const int4*>(s_ids + j);
      before += (v.x == id) + (j + 1 < i && v.y == id) + (j + 2 < i && v.z == id) +
                (j + 3 < i && v.w == id);
    }
    first = before % kGroup == 0;
  }
  const uint32_t m = __ballot_sync(0xffffffffu, first);
  if (lane == 0 && warp < kFewTokens / 32) s_first[warp] = m;
  __syncthreads();
  int at = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kFewTokens / 32; ++w) {
    const int n = __popc(s_first[w]);
    at += w < warp ? n : w == warp ? __popc(s_first[w] & ((1u << lane) - 1)) : 0;
    all += n;
  }
  if (first) s_group[at] = make_int2(i, before);
  __syncthreads();
  return all;
}

template <typename T, typename YT, int CTAS, int WARPS, bool ANY>
__global__ void __launch_bounds__(32 * WARPS, 16 / WARPS) adapters_few(AdapterArgs p) {
  __shared__ __align__(16) int s_ids[kFewTokens];
  __shared__ int2 s_group[kFewTokens];
  __shared__ int s_token[kGroup];
  __shared__ float s_down[kGroup];
  __shared__ __align__(16) FewShared<T, WARPS> s_mem;
  __shared__ float s_part[kGroup * kMaxRank];
  cg::cluster_group cluster = cg::this_cluster();
  const int cta = cluster.block_rank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int o_per = (p.n_out + 32 * CTAS - 1) / (32 * CTAS) * 32;
  const int o0 = min(cta * o_per, p.n_out), o1 = min(o0 + o_per, p.n_out);
  const int2 inner = inner_share(0, p.n_in, cta, CTAS);
  const int k0 = inner.x, k1 = inner.y;
  const int groups = few_groups<WARPS>(p, s_ids, s_group);
  // every CTA of a cluster goes through the same groups
  for (int q = blockIdx.x / CTAS; q < groups; q += gridDim.x / CTAS) {
    const int2 group = s_group[q];
    const int slot = s_ids[group.x];
    const int rank = slot >= 0 ? rank_of(p, slot) : 0;
    // the group's tokens: the first of them and the next seven of its slot
    int n_tokens = 0;
    for (int i = group.x / 32 * 32; i < p.n_tokens && n_tokens < kGroup; i += 32) {
      const int at = i + lane;
      const uint32_t m =
          __ballot_sync(0xffffffffu, at >= group.x && at < p.n_tokens && s_ids[at] == slot);
      const int place = n_tokens + __popc(m & ((1u << lane) - 1));
      if (warp == 0 && (m >> lane & 1) && place < kGroup) s_token[place] = at;
      n_tokens += __popc(m);
    }
    n_tokens = min(n_tokens, kGroup);
    if (rank == 0) {
      __syncthreads();
      for (int k = 0; k < n_tokens; ++k) copy_base<YT>(p, s_token[k], o0, o1);
      __syncthreads();
      continue;
    }
    const T* a = static_cast<const T*>(p.a) + (int64_t)slot * p.rank * p.n_in;
    const T* b = static_cast<const T*>(p.b) + (int64_t)slot * p.n_out * p.rank;
    __syncthreads();
    // (memory is at work on all of A's share before the first load waits)
    for (int i = threadIdx.x; i < rank; i += 32 * WARPS)
      prefetch_bulk(a + (int64_t)i * p.n_in + k0, (k1 - k0) * (int64_t)sizeof(T));
    const T* x = static_cast<const T*>(p.x) + s_token[min(lane >> 2, n_tokens - 1)] * p.xs;
    if (rank <= 16)
      few_shrink<T, 1, WARPS, ANY>(p, a, rank, 0, x, k0, k1, s_mem.warps, s_part);
    else if (rank <= 32)
      few_shrink<T, 2, WARPS, ANY>(p, a, rank, 0, x, k0, k1, s_mem.warps, s_part);
    else
      for (int j0 = 0; j0 < rank; j0 += 64)
        few_shrink<T, 4, WARPS, ANY>(p, a, rank, j0, x, k0, k1, s_mem.warps, s_part);
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    // (any earlier, B would take its share of the memory from A)
    const int64_t share = (int64_t)(o1 - o0) * p.rank;
    if (lane == 0)
      prefetch_bulk(b + (int64_t)o0 * p.rank + share * warp / WARPS,
                    (share * (warp + 1) / WARPS - share * warp / WARPS) * (int)sizeof(T));
    if (p.base && (int)threadIdx.x < n_tokens)
      prefetch_bulk(static_cast<const YT*>(p.base) + s_token[threadIdx.x] * p.bs + o0,
                    (o1 - o0) * (int64_t)sizeof(YT));
    const int nk = (rank + 31) / 32;
    // a step's base and first 32 columns of B: two steps are under way at a time
    struct Step {
      uint4 w[4];
      Pack<YT, 4> v[1][2];
    } now, then;
    const auto load_step = [&](Step& s, int o) {
      if (o >= o1) return;
      load_b(p, b, rank, 0, o, s.w);
      load_base<YT, 1>(p, s_token, n_tokens, o, s.v);
    };
    int o = o0 + 32 * warp;
    load_step(now, o);
    const float scale = p.scales ? p.scales[slot] : 1.f;
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp < n_tokens) {  // a warp per token: its h over the cluster's shares
      float h[kMaxRank / 32];
#pragma unroll
      for (int i = 0; i < kMaxRank / 32; ++i) {
        h[i] = 0.f;
        if (i < nk && i * 32 + lane < rank) {
          float part[CTAS];
#pragma unroll
          for (int c = 0; c < CTAS; ++c)
            part[c] = cluster.map_shared_rank(s_part, c)[warp * kMaxRank + i * 32 + lane];
#pragma unroll
          for (int c = 0; c < CTAS; ++c) h[i] += part[c];
        }
      }
      const float down = split_terms<T>(h, nk, s_mem.h + warp * kPitch, kGroup * kPitch);
      if (lane == 0) s_down[warp] = down;
    } else if (warp < kGroup) {  // columns of the matrix instruction that no token has
      for (int k = 0; k < Terms<T>::n; ++k)
        for (int j = lane; j < kPitch; j += 32)
          s_mem.h[(k * kGroup + warp) * kPitch + j] = from_f32<T>(0.f);
    }
    __syncthreads();
    // the others may still read this CTA's share: its memory changes after them
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    const auto do_step = [&](Step& s, int o) {
      float acc[2][1][4] = {};
      expand<T, 1>(s.w, s_mem.h, kPitch, kGroup * kPitch, acc);
      for (int k = 1; k < nk; ++k) {
        load_b(p, b, rank, k, o, s.w);
        expand<T, 1>(s.w, s_mem.h + 32 * k, kPitch, kGroup * kPitch, acc);
      }
      finish<YT, 1>(p, s_token, n_tokens, s_down, scale, o, s.v, acc);
    };
    while (o < o1) {
      load_step(then, o + 32 * WARPS);
      do_step(now, o);
      o += 32 * WARPS;
      if (o >= o1) break;
      load_step(now, o + 32 * WARPS);
      do_step(then, o);
      o += 32 * WARPS;
    }
    __syncthreads();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  }
}

// Nothing to add: a CTA per token.
template <typename YT>
__global__ void __launch_bounds__(kThreads) adapters_copy(AdapterArgs p) {
  copy_base<YT>(p, blockIdx.x, 0, p.n_out);
}

// --------------------------------------------------- many tokens (prompts)
// Tokens are first sorted by slot and cut into tiles of one slot's tokens;
// then A x per tile, by a cluster whose CTAs take shares of the inner range
// and meet in distributed shared memory; then y per tile and share of the
// columns.
constexpr int kTile = 64;
constexpr int kSortThreads = 1024;
constexpr int kMaxSplit = 8;  // shares of the inner range: a portable cluster

__global__ void __launch_bounds__(kSortThreads) adapters_sort(AdapterArgs p) {
  extern __shared__ int s_count[];  // per slot, the tokens without one last
  __shared__ int2 s_warp[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n = p.n_slots + 1;
  pdl_launch_dependents();
  for (int i = threadIdx.x; i < n; i += kSortThreads) s_count[i] = 0;
  __syncthreads();
  const auto slot_at = [&](int i) {
    const int s = p.ids[i];
    return s >= 0 && s < p.n_slots ? s : p.n_slots;
  };
  // one atomic for the lanes of a warp that share a slot
  const int rounds = (p.n_tokens + kSortThreads - 1) / kSortThreads;
#pragma unroll 4
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
    // in whatever order the warps come: each token's sums are added in one
    // order, whichever tile it is in (shrink)
    if (s >= 0) p.perm[base + __popc(same & ((1u << lane) - 1))] = i;
  }
}

// The warps take shares of the CTA's inner range, each for all of the tile's
// tokens (8 NT of them at most): A is read once per tile. Their sums meet in
// s_warp, [warp][token][16 MT + 1], and go to s_sum, [token][sum_pitch].
template <typename T, int MT, int NT, bool ANY>
__device__ __forceinline__ void tile_shrink(const AdapterArgs& p, const T* a, int rank, int j0,
                                            const int32_t* tokens, int n_tokens, int k0, int k1,
                                            float* s_warp, float* s_sum, int sum_pitch) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const T* x[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n)
    x[n] = static_cast<const T*>(p.x) + tokens[min(8 * n + g, n_tokens - 1)] * p.xs;
  const int2 mine = inner_share(k0, k1, warp, kWarps);
  float acc[MT][NT][4] = {};
  shrink<T, MT, NT, kTile / 8, ANY>(p, a, rank, j0, x, mine.x, mine.y, acc);
  constexpr int kWide = 16 * MT + 1;
  float* out = s_warp + warp * 8 * NT * kWide;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        out[(8 * n + 2 * t + (e & 1)) * kWide + 16 * m + g + 8 * (e >> 1)] = acc[m][n][e];
  __syncthreads();
  for (int i = threadIdx.x; i < n_tokens * 16 * MT; i += kThreads) {
    const int token = i / (16 * MT), j = i % (16 * MT);
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += s_warp[(w * 8 * NT + token) * kWide + j];
    s_sum[token * sum_pitch + j0 + j] = v;
  }
  __syncthreads();
}

// tile_shrink over a slot's rank, by blocks of 64.
template <typename T, bool WIDE, int NT, bool ANY>
__device__ __forceinline__ void tile_shrink_all(const AdapterArgs& p, const T* a, int rank,
                                                const int32_t* tokens, int n_tokens, int k0,
                                                int k1, float* s_warp, float* s_sum, int pitch) {
  if (rank <= 16)
    tile_shrink<T, 1, NT, ANY>(p, a, rank, 0, tokens, n_tokens, k0, k1, s_warp, s_sum, pitch);
  else if (rank <= 32)
    tile_shrink<T, 2, NT, ANY>(p, a, rank, 0, tokens, n_tokens, k0, k1, s_warp, s_sum, pitch);
  if constexpr (WIDE)
    if (rank > 32)
      for (int j0 = 0; j0 < rank; j0 += 64)
        tile_shrink<T, 4, NT, ANY>(p, a, rank, j0, tokens, n_tokens, k0, k1, s_warp, s_sum, pitch);
}

// Columns of a token's sums: whole blocks of 16 MT, on other banks.
constexpr int sum_pitch_of(int rank) {
  return (rank <= 16 ? 16 : rank <= 32 ? 32 : (rank + 63) / 64 * 64) + 4;
}
// Floats of the warps' sums, for tiles of kTile tokens.
constexpr int warp_sums_of(int rank) {
  return kWarps * kTile * ((rank <= 16 ? 16 : rank <= 32 ? 32 : 64) + 1);
}

template <typename T, bool WIDE, bool ANY>  // WIDE: ranks above 32
__global__ void __launch_bounds__(kThreads, 1) adapters_shrink(AdapterArgs p) {
  extern __shared__ float s_dyn_sum[];  // kTile x sum_pitch_of(p.rank), then the warps' sums
  pdl_launch_dependents();
  cg::cluster_group cluster = cg::this_cluster();
  const int split = blockIdx.x % p.k_split;
  const int2 inner = inner_share(0, p.n_in, split, p.k_split);
  const int k0 = inner.x, k1 = inner.y, pitch = sum_pitch_of(p.rank);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float* s_sum = s_dyn_sum;
  float* s_warp = s_sum + kTile * pitch;
  pdl_wait();
  const int n_tiles = *p.n_tiles;
  // every CTA of a cluster goes through the same tiles
  for (int i = blockIdx.x / p.k_split; i < n_tiles; i += gridDim.x / p.k_split) {
    const int4 tile = p.tiles[i];
    const int rank = tile.x < 0 ? 0 : rank_of(p, tile.x);
    if (rank == 0) continue;
    const T* a = static_cast<const T*>(p.a) + (int64_t)tile.x * p.rank * p.n_in;
    if (tile.z > 32)
      tile_shrink_all<T, WIDE, 8, ANY>(p, a, rank, p.perm + tile.y, tile.z, k0, k1, s_warp, s_sum, pitch);
    else if (tile.z > 8)
      tile_shrink_all<T, WIDE, 4, ANY>(p, a, rank, p.perm + tile.y, tile.z, k0, k1, s_warp, s_sum, pitch);
    else
      tile_shrink_all<T, WIDE, 1, ANY>(p, a, rank, p.perm + tile.y, tile.z, k0, k1, s_warp, s_sum, pitch);
    cluster.sync();
    // a warp per token: its h over the cluster's shares, as 16-bit terms
    const int nk = (rank + 31) / 32;
    for (int k = split * kWarps + warp; k < tile.z; k += p.k_split * kWarps) {
      float h[kMaxRank / 32];
#pragma unroll
      for (int q = 0; q < kMaxRank / 32; ++q) {
        h[q] = 0.f;
        if (q < nk && q * 32 + lane < rank) {
          float part[kMaxSplit];
#pragma unroll
          for (int c = 0; c < kMaxSplit; ++c)
            part[c] = c < p.k_split ? cluster.map_shared_rank(s_sum, c)[k * pitch + q * 32 + lane]
                                    : 0.f;
#pragma unroll
          for (int c = 0; c < kMaxSplit; ++c) h[q] += part[c];
        }
      }
      T* out = static_cast<T*>(p.terms) + (int64_t)(tile.y + k) * Terms<T>::n * p.term_pitch;
      const float down = split_terms<T>(h, nk, out, p.term_pitch);
      if (lane == 0) p.downs[tile.y + k] = down;
    }
    cluster.sync();  // no CTA changes its sums or leaves while another reads them
  }
}

// Elements from token to token in shared memory: 64 bytes past a multiple of
// 128, so that the two rows of a quarter-warp's 16-byte loads do not meet.
template <typename T>
__host__ __device__ constexpr int pitch_of(int row) {
  return row * (int)sizeof(T) % 128 == 64 ? row : row + 64 / (int)sizeof(T);
}

// base's steps are on their way into shared memory, each lane's own places,
// while the step before is multiplied and stored.
constexpr int kBaseStages = 2;

template <typename T, typename YT>
__global__ void __launch_bounds__(kThreads, 2) adapters_expand(AdapterArgs p) {
  extern __shared__ __align__(16) unsigned char s_dyn[];
  T* s_h = reinterpret_cast<T*>(s_dyn);  // [token][term][term_pitch]
  __shared__ int s_token[kTile];
  __shared__ float s_down[kTile];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = Terms<T>::n * p.term_pitch, pitch = pitch_of<T>(row);
  using P = Pack<YT, 4>;
  // [stage][warp][8 places][lane]
  P* ring = reinterpret_cast<P*>(s_dyn + (size_t)kTile * pitch * sizeof(T)) + warp * 256 + lane;
  const bool async = p.base && p.vec_y;
  pdl_wait();
  // (tile, 128 columns) steps in equal contiguous shares
  const int per_tile = (p.n_out + 127) / 128;
  const int64_t steps = (int64_t)*p.n_tiles * per_tile;
  int64_t step = steps * blockIdx.x / gridDim.x;
  const int64_t end = steps * (blockIdx.x + 1) / gridDim.x;
  while (step < end) {
    const int4 tile = p.tiles[step / per_tile];
    const int from = (int)(step % per_tile), to = (int)min((int64_t)per_tile, from + end - step);
    step += to - from;
    const int o0 = 128 * from, o1 = min(128 * to, p.n_out);
    const int rank = tile.x < 0 ? 0 : rank_of(p, tile.x);
    if (rank == 0) {
      for (int k = 0; k < tile.z; ++k) copy_base<YT>(p, p.perm[tile.y + k], o0, o1);
      continue;
    }
    const int nk = (rank + 31) / 32;
    __syncthreads();  // the last tile's terms are done with
    if ((int)threadIdx.x < kTile) {
      const int k = tile.y + min((int)threadIdx.x, tile.z - 1);
      s_token[threadIdx.x] = p.perm[k];
      s_down[threadIdx.x] = p.downs[k];
    }
    // terms of the tile's tokens (places past them repeat the last token's)
    const T* terms = static_cast<const T*>(p.terms) + (int64_t)tile.y * row;
    for (int k = threadIdx.x; k < kTile * row / 8; k += kThreads) {
      const int token = k / (row / 8), c = k % (row / 8) * 8;
      *reinterpret_cast<uint4*>(s_h + token * pitch + c) =
          *reinterpret_cast<const uint4*>(terms + (int64_t)min(token, tile.z - 1) * row + c);
    }
    __syncthreads();
    const T* b = static_cast<const T*>(p.b) + (int64_t)tile.x * p.n_out * p.rank;
    const float scale = p.scales ? p.scales[tile.x] : 1.f;
    // two halves of the tile's tokens times four blocks of 32 columns, or
    // eight blocks where the tile has half its tokens at most
    const int halves = tile.z > 32 ? 2 : 1, half = warp % halves, n_tokens = tile.z - 32 * half;
    const T* h = s_h + 32 * half * pitch;
    const int* tokens = s_token + 32 * half;
    const int stride = 32 * kWarps / halves;
    const auto fetch = [&](int o, int stage) {
      if (o < o1) {
        const int g = lane & 7, t = lane >> 3, c = o + 4 * g;
        const YT* at = static_cast<const YT*>(p.base) + c;
        P* to = ring + stage * kWarps * 256;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int i = 8 * (k >> 1) + 2 * t + (k & 1);
          if (i < n_tokens && c < p.n_out)
            copy_async<sizeof(P)>(to + 32 * k, at + tokens[i] * p.bs);
        }
      }
      copy_commit();
    };
    int o = o0 + 32 * (warp / halves), stage = 0;
    if (async) {
#pragma unroll
      for (int k = 0; k < kBaseStages - 1; ++k) fetch(o + k * stride, k);
    }
    uint4 w[4];
    if (o < o1) load_b(p, b, rank, 0, o, w);
    for (; o < o1; o += stride) {
      if (async) fetch(o + (kBaseStages - 1) * stride, (stage + kBaseStages - 1) % kBaseStages);
      float acc[2][4][4] = {};
      expand<T, 4>(w, h, pitch, p.term_pitch, acc);
      for (int k = 1; k < nk; ++k) {
        load_b(p, b, rank, k, o, w);
        expand<T, 4>(w, h + 32 * k, pitch, p.term_pitch, acc);
      }
      if (o + stride < o1) load_b(p, b, rank, 0, o + stride, w);
      P v[4][2];
      if (async) {
        copy_wait<kBaseStages - 1>();
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k >> 1][k & 1] = ring[stage * kWarps * 256 + 32 * k];
        stage = (stage + 1) % kBaseStages;
      } else {
        load_base<YT, 4>(p, tokens, n_tokens, o, v);
      }
      finish<YT, 4>(p, tokens, n_tokens, s_down + 32 * half, scale, o, v, acc);
    }
  }
}

constexpr int kSms = 152;
constexpr int kMaxTokens = 1 << 27, kMaxWidth = 1 << 30;  // (32-bit grids and columns)

int64_t round_up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

// Workspace of the sorted path: tile count, tiles, sorted tokens, h.
struct Workspace {
  int64_t tiles, perm, downs, terms, bytes;
  int max_tiles, k_split, term_pitch;
};

Workspace workspace_of(int n_tokens, int n_slots, int rank) {
  Workspace w{};
  if (n_tokens <= kFewTokens || n_slots == 0 || rank == 0) return w;
  w.max_tiles = n_tokens / kTile + (n_slots + 1 < n_tokens ? n_slots + 1 : n_tokens);
  // as many CTAs as one wave holds, with tiles as full as can be (400 tokens
  // of 12288 x 12288 at rank 32: 31 us, unsplit 66; 2048 tokens 69, split for
  // two waves 81)
  const int tiles = (n_tokens + kTile - 1) / kTile;
  w.k_split = 1;
  while (w.k_split < kMaxSplit && tiles * 2 * w.k_split <= kSms) w.k_split *= 2;
  w.term_pitch = (rank + 31) / 32 * 32;
  w.tiles = 16;
  w.perm = round_up(w.tiles + 16ll * w.max_tiles, 128);
  w.downs = round_up(w.perm + 4ll * n_tokens, 128);
  w.terms = round_up(w.downs + 4ll * n_tokens, 128);
  w.bytes = w.terms + 2ll * Terms<__nv_bfloat16>::n * w.term_pitch * n_tokens;
  return w;
}

int launch_cluster(const void* fn, int grid, int block, size_t smem, int cluster, bool pdl,
                   cudaStream_t st, void** args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelExC(&cfg, fn, args) == cudaSuccess ? 0 : -1;
}

template <typename T, typename YT>
spmv_status run_few(AdapterArgs& p, cudaStream_t st) {
  void* args[] = {&p};
  // groups, at most: each slot's tokens in eights, and so those without one
  const int most = p.n_tokens / kGroup + p.n_slots + 1;
  const int groups = p.n_tokens < most ? p.n_tokens : most;
  int e;
  // clusters of 16 while there are SMs for all of them (one token of 12288 x
  // 12288 at rank 16: 10.4 us, clusters of 8: 14.2)
  if (groups <= 9) {
    const void* fn = p.vec_in ? reinterpret_cast<const void*>(&adapters_few<T, YT, 16, 16, false>)
                              : reinterpret_cast<const void*>(&adapters_few<T, YT, 16, 16, true>);
    const spmv_status leave =
        status_of(cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    if (leave != SPMV_OK) return leave;
    e = launch_cluster(fn, groups * 16, 512, 0, 16, false, st, args);
  } else {  // at most two waves of two CTAs per SM
    const void* fn = p.vec_in ? reinterpret_cast<const void*>(&adapters_few<T, YT, 8, 8, false>)
                              : reinterpret_cast<const void*>(&adapters_few<T, YT, 8, 8, true>);
    const int clusters = groups < 76 ? groups : 76;
    e = launch_cluster(fn, clusters * 8, 256, 0, 8, false, st, args);
  }
  return status_of_launch(e);
}

template <typename T, typename YT>
spmv_status run_many(AdapterArgs& p, cudaStream_t st) {
  const size_t sort_smem = (size_t)(p.n_slots + 1) * 4;
  const size_t shrink_smem = ((size_t)kTile * sum_pitch_of(p.rank) + warp_sums_of(p.rank)) * 4;
  const size_t expand_smem = (size_t)kTile * pitch_of<T>(Terms<T>::n * p.term_pitch) * sizeof(T) +
                             (size_t)kBaseStages * kThreads * 8 * sizeof(Pack<YT, 4>);
  const bool wide = p.rank > 32;
  const void* shrink_fn =
      p.vec_in ? (wide ? reinterpret_cast<const void*>(&adapters_shrink<T, true, false>)
                       : reinterpret_cast<const void*>(&adapters_shrink<T, false, false>))
               : (wide ? reinterpret_cast<const void*>(&adapters_shrink<T, true, true>)
                       : reinterpret_cast<const void*>(&adapters_shrink<T, false, true>));
  const void* expand_fn = reinterpret_cast<const void*>(&adapters_expand<T, YT>);
  if (!allow_smem(reinterpret_cast<const void*>(&adapters_sort), sort_smem) ||
      !allow_smem(shrink_fn, shrink_smem) || !allow_smem(expand_fn, expand_smem))
    return SPMV_ERR_CUDA;
  const spmv_status sorted = launch(adapters_sort, dim3(1), kSortThreads, sort_smem, st, p);
  if (sorted != SPMV_OK) return sorted;
  void* args[] = {&p};
  const int most = resident_clusters(shrink_fn, p.k_split, kThreads, shrink_smem);
  if (most == 0) return SPMV_ERR_CUDA;
  const int clusters = p.max_tiles < most ? p.max_tiles : most;
  // (two CTAs per SM where the terms of a large rank leave room for them)
  const int64_t wave = expand_smem <= 112 * 1024 ? 2 * kSms : kSms;
  const int64_t steps = (int64_t)p.max_tiles * ((p.n_out + 127) / 128);
  int e = launch_cluster(shrink_fn, clusters * p.k_split, kThreads, shrink_smem, p.k_split, true,
                         st, args);
  if (e == 0)
    e = launch_pdl(expand_fn, (int)(steps < wave ? steps : wave), kThreads, expand_smem, st, args);
  return status_of_launch(e);
}

template <typename T, typename YT>
spmv_status run(AdapterArgs& p, cudaStream_t st) {
  if (p.n_slots == 0) {
    if (p.base == p.y) return SPMV_OK;
    return launch(adapters_copy<YT>, dim3((unsigned)p.n_tokens), kThreads, 0, st, p);
  }
  return p.n_tokens <= kFewTokens ? run_few<T, YT>(p, st) : run_many<T, YT>(p, st);
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
  if (p.vec_in && n_in % 16 == 0 && aligned_to(x, 32) && aligned_to(a, 32) &&
      (n_tokens == 1 || x_stride % 16 == 0))
    p.vec_in = 2;
  p.vec_b = rank % 8 == 0 && aligned_to(b, 16)  ? 1
            : rank % 4 == 0 && aligned_to(b, 8) ? 8
            : rank % 2 == 0 && aligned_to(b, 4) ? 4
                                                : 0;
  p.vec_y = n_out % 4 == 0 && rows_aligned(y, n_tokens, y_stride, ysz, 4) &&
            (!base || rows_aligned(base, n_tokens, base_stride, ysz, 4));
  if (w.bytes > 0) {
    char* at = static_cast<char*>(workspace);
    p.n_tiles = reinterpret_cast<int32_t*>(at);
    p.tiles = reinterpret_cast<int4*>(at + w.tiles);
    p.perm = reinterpret_cast<int32_t*>(at + w.perm);
    p.downs = reinterpret_cast<float*>(at + w.downs);
    p.terms = at + w.terms;
    p.max_tiles = w.max_tiles, p.k_split = w.k_split, p.term_pitch = w.term_pitch;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SPMV_F16)
    return y_dtype == SPMV_F32 ? run<__half, float>(p, st) : run<__half, __half>(p, st);
  return y_dtype == SPMV_F32 ? run<__nv_bfloat16, float>(p, st)
                             : run<__nv_bfloat16, __nv_bfloat16>(p, st);
}
