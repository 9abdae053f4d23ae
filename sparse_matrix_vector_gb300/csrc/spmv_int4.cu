// Products with 4-bit weights and group scales (spmv_int4_run):
//   y_t = base_t + W x_t,  W[o, i] = scale[o, i / group] * (q[o, i] - zero[o, i / group]),
// for a few tokens t. Bound by reading the packed weights once. They become
// exact small integers in x's 16-bit type (bits or-ed into the mantissa of
// 1024 or 128, less 1024 or 128 plus the zero point) that go through the
// warp-level matrix instruction (16 weights' rows x 8 tokens x 16 columns,
// fp32 sums); a group's sum is scaled in fp32 once it is whole, so nothing is
// rounded before the products' own sums.
//
// The order of the columns within a sum is free as long as both operands agree
// on it: a 32-bit word of 8 columns gives two instructions' worth of one
// lane's share, in the pairs (0, 4), (1, 5), (2, 6), (3, 7) that masks take out
// of it, and x is taken in the same pairs.
#include <climits>
#include <type_traits>

#include "spmv_device.cuh"
#include "spmv_types.cuh"

namespace spmv {
namespace {

constexpr int kWarpsInt4 = 8;
constexpr int kStep = 128;             // columns that a warp takes at a time
constexpr int kStepBytes = kStep / 2;
constexpr int kRing = 4;               // steps of weights in shared memory

struct Int4Args {
  int n_tokens, n_in, n_out, group, groups;
  const void* x;
  int64_t xs;
  const uint8_t* w;
  int64_t ws;
  const void* scales;
  const uint8_t* zeros;
  const void* base;
  int64_t bs;
  void* y;
  int64_t ys;
  int group_shift;  // log2(group), or 31: one group
  bool scales_f32, vec_x;
};

template <typename T>
__device__ __forceinline__ void mma_int4(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (w & mask) | bits
__device__ __forceinline__ uint32_t take_bits(uint32_t w, uint32_t mask, uint32_t bits) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(bits));
  return r;
}

// What turns 8 nibbles into exact integers less a zero point.
template <typename T>
struct Unpack;
template <>
struct Unpack<__half> {
  uint32_t low, high;  // -(1024 + z) and -(64 + z), twice
  __device__ __forceinline__ void set(uint32_t z) {
    low = (0xe400u + z) * 0x10001u;
    high = (0xd400u + (z << 4)) * 0x10001u;
  }
  // words of the pairs (0, 4), (1, 5), (2, 6), (3, 7)
  __device__ __forceinline__ void run(uint32_t w, uint32_t (&r)[4]) const {
    const __half2 lo = reinterpret_cast<const __half2&>(low), hi = reinterpret_cast<const __half2&>(high);
    const __half2 sixteenth = __half2half2(__ushort_as_half(0x2c00));
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t v = w >> (8 * k);
      // 1024 + n, and 1024 + 16 n = 16 (64 + n)
      const uint32_t a = take_bits(v, 0x000f000fu, 0x64006400u), b = take_bits(v, 0x00f000f0u, 0x64006400u);
      const __half2 p = __hadd2(reinterpret_cast<const __half2&>(a), lo);
      const __half2 q = __hfma2(reinterpret_cast<const __half2&>(b), sixteenth, hi);
      r[2 * k] = reinterpret_cast<const uint32_t&>(p);
      r[2 * k + 1] = reinterpret_cast<const uint32_t&>(q);
    }
  }
};
template <>
struct Unpack<__nv_bfloat16> {
  uint32_t low;  // -(128 + z), twice
  __device__ __forceinline__ void set(uint32_t z) { low = (0xc300u + z) * 0x10001u; }
  __device__ __forceinline__ void run(uint32_t w, uint32_t (&r)[4]) const {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t a = take_bits(w >> (4 * k), 0x000f000fu, 0x43004300u);
      const __nv_bfloat162 p = __hadd2(reinterpret_cast<const __nv_bfloat162&>(a),
                                       reinterpret_cast<const __nv_bfloat162&>(low));
      r[k] = reinterpret_cast<const uint32_t&>(p);
    }
  }
};

// Where piece p (16 bytes) of row r stands in a stage: rows of 64 bytes whose
// pieces are exchanged so that reads of 4, 8 or 16 bytes by 8 rows x 4 lanes
// meet every bank once.
__device__ __forceinline__ int piece_at(int r, int p) {
  return r * kStepBytes + ((p ^ (((r >> 1) & 1) << 1 | ((r >> 2) & 1))) << 4);
}

// 16 bytes at p of which `left` are inside the row (the others zero), any
// alignment: the two 16-byte granules around them, shifted into place.
__device__ __forceinline__ uint4 load_piece(const uint8_t* p, int left) {
  uint4 r = make_uint4(0, 0, 0, 0);
  if (left <= 0) return r;
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  const uint4* g = reinterpret_cast<const uint4*>(at & ~uintptr_t(15));
  const int skip = (int)(at & 15);
  const uint4 a = __ldg(g);
  uint4 b = make_uint4(0, 0, 0, 0);
  if (skip + min(left, 16) > 16) b = __ldg(g + 1);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t v[5];
#pragma unroll
  for (int k = 0; k < 5; ++k) {
    const uint32_t e = skip & 4 ? (k + 1 < 8 ? w[k + 1] : 0) : w[k];
    const uint32_t f = skip & 4 ? (k + 3 < 8 ? w[k + 3] : 0) : w[k + 2];
    v[k] = skip & 8 ? f : e;
  }
  const uint32_t bits = 8 * (skip & 3);
  r = make_uint4(__funnelshift_r(v[0], v[1], bits), __funnelshift_r(v[1], v[2], bits),
                 __funnelshift_r(v[2], v[3], bits), __funnelshift_r(v[3], v[4], bits));
  return r;  // (bytes behind the row meet zeros of x)
}

// 8 elements of x at p, `left` of them inside the row (the others zero).
template <typename T>
__device__ __forceinline__ uint4 load_x(const T* p, int left, bool vec) {
  if (vec && left >= 8) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t e[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    e[k] = 0;
    if (k < left) e[k] = __ldg(reinterpret_cast<const unsigned short*>(p) + k);
  }
  return make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
}

// A CTA: 16 MT rows of W for 8 NT tokens, the columns split over its warps. SEG:
// columns whose sums are scaled together (a group, or a step of a longer one).
template <typename T, typename YT, int MT, int NT, int SEG, bool ALIGNED>
__global__ void __launch_bounds__(kWarpsInt4 * 32) int4_rows(Int4Args a) {
  extern __shared__ __align__(16) unsigned char s_int4[];
  constexpr int kRows = 16 * MT, kStage = kRows * kStepBytes, kWords = SEG / 32;
  constexpr int kPieces = kStage / 16 / 32;  // of a lane
  const int me = threadIdx.x, warp = me >> 5, lane = me & 31, g = lane >> 2, q = lane & 3;
  const int row0 = blockIdx.x * kRows, token0 = blockIdx.y * 8 * NT;
  const int row_bytes = (a.n_in + 1) / 2;
  const int steps = (a.n_in + kStep - 1) / kStep;
  const int begin = (int)((int64_t)steps * warp / kWarpsInt4), end = (int)((int64_t)steps * (warp + 1) / kWarpsInt4);
  unsigned char* ring = s_int4 + warp * kRing * kStage;

  // this lane's pieces of a step: rows (lane / 4) + 8 k, piece lane % 4
  const uint8_t* src[kPieces];
#pragma unroll
  for (int k = 0; k < kPieces; ++k)
    src[k] = a.w + (int64_t)min(row0 + g + 8 * k, a.n_out - 1) * a.ws;
  const auto fetch = [&](int step) {
    if (step < end) {
      const int at = step * kStepBytes + q * 16;
      unsigned char* to = ring + (step & (kRing - 1)) * kStage;
#pragma unroll
      for (int k = 0; k < kPieces; ++k) {
        unsigned char* dst = to + piece_at(g + 8 * k, q);
        if constexpr (ALIGNED) {
          const int bytes = max(0, min(16, row_bytes - at));
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)),
                       "l"(src[k] + (bytes > 0 ? at : 0)), "r"(bytes)
                       : "memory");
        } else {
          *reinterpret_cast<uint4*>(dst) = load_piece(src[k] + at, row_bytes - at);
        }
      }
    }
    if constexpr (ALIGNED) copy_commit();
  };

  const T* x[NT];
  bool has[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = token0 + 8 * n + g;
    has[n] = t < a.n_tokens;
    x[n] = static_cast<const T*>(a.x) + (has[n] ? (int64_t)t * a.xs : 0);
  }
  // scales and zero points of this lane's rows (2 m + h: row 16 m + 8 h + g)
  float scale[2][2 * MT];
  uint32_t zero[2][2 * MT];
  const auto group_of = [&](int col) { return min(col >> a.group_shift, a.groups - 1); };
  const auto load_scales = [&](int col, float (&s)[2 * MT], uint32_t (&z)[2 * MT]) {
    const int k = group_of(col);
#pragma unroll
    for (int r = 0; r < 2 * MT; ++r) {
      const int64_t at = (int64_t)min(row0 + 8 * r + g, a.n_out - 1) * a.groups + k;
      s[r] = a.scales_f32 ? __ldg(static_cast<const float*>(a.scales) + at)
                          : to_f32(static_cast<const T*>(a.scales)[at]);
      z[r] = a.zeros ? __ldg(a.zeros + at) & 15u : 8u;
    }
  };

  float acc[MT][NT][4] = {};
#pragma unroll
  for (int k = 0; k < kRing - 1; ++k) fetch(begin + k);
  if (begin < end) load_scales(begin * kStep, scale[0], zero[0]);
  int now = 0;
  for (int step = begin; step < end; ++step) {
    if constexpr (ALIGNED) copy_wait<kRing - 2>();
    __syncwarp();
    const unsigned char* stage = ring + (step & (kRing - 1)) * kStage;
    fetch(step + kRing - 1);
#pragma unroll
    for (int seg = 0; seg < kStep / SEG; ++seg) {
      const int col0 = step * kStep + seg * SEG;
      // the next segment's, while this one is computed
      if (seg + 1 < kStep / SEG || step + 1 < end) {
        if (now == 0)
          load_scales(col0 + SEG, scale[1], zero[1]);
        else
          load_scales(col0 + SEG, scale[0], zero[0]);
      }
      float s_now[2 * MT];
      Unpack<T> un[2 * MT];
#pragma unroll
      for (int r = 0; r < 2 * MT; ++r) {
        s_now[r] = now == 0 ? scale[0][r] : scale[1][r];
        un[r].set(now == 0 ? zero[0][r] : zero[1][r]);
      }
      now ^= 1;
      float part[MT][NT][4] = {};
      // this lane's words of the segment: columns col0 + q * 8 kWords + 8 w
      uint32_t w[2 * MT][kWords];
      const int byte = seg * (SEG / 2) + q * 4 * kWords;
#pragma unroll
      for (int r = 0; r < 2 * MT; ++r) {
        const unsigned char* at = stage + piece_at(g + 8 * r, byte >> 4) + (byte & 15);
        if constexpr (kWords == 4) {
          const uint4 v = *reinterpret_cast<const uint4*>(at);
          w[r][0] = v.x, w[r][1] = v.y, w[r][2] = v.z, w[r][3] = v.w;
        } else if constexpr (kWords == 2) {
          const uint2 v = *reinterpret_cast<const uint2*>(at);
          w[r][0] = v.x, w[r][1] = v.y;
        } else {
          w[r][0] = *reinterpret_cast<const uint32_t*>(at);
        }
      }
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
        const int col = col0 + q * 8 * kWords + 8 * k;
        uint32_t b[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 v = load_x(x[n] + col, has[n] ? a.n_in - col : 0, a.vec_x);
          b[n][0] = __byte_perm(v.x, v.z, 0x5410);
          b[n][1] = __byte_perm(v.x, v.z, 0x7632);
          b[n][2] = __byte_perm(v.y, v.w, 0x5410);
          b[n][3] = __byte_perm(v.y, v.w, 0x7632);
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint32_t lo[4], hi[4];
          un[2 * m].run(w[2 * m][k], lo);
          un[2 * m + 1].run(w[2 * m + 1][k], hi);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_int4<T>(part[m][n], lo[0], hi[0], lo[1], hi[1], b[n][0], b[n][1]);
            mma_int4<T>(part[m][n], lo[2], hi[2], lo[3], hi[3], b[n][2], b[n][3]);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[m][n][k] += s_now[2 * m + (k >> 1)] * part[m][n][k];
    }
    __syncwarp();  // (all lanes are done with the stage before it is filled again)
  }
  if constexpr (ALIGNED) copy_wait<0>();
  __syncthreads();

  // the warps' sums, joined in their order
  constexpr int kPitch = kRows + 1;
  float* sums = reinterpret_cast<float*>(s_int4);
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        sums[(warp * 8 * NT + 8 * n + 2 * q + (k & 1)) * kPitch + 16 * m + 8 * (k >> 1) + g] = acc[m][n][k];
  __syncthreads();
  for (int e = me; e < kRows * 8 * NT; e += kWarpsInt4 * 32) {
    const int r = e % kRows, n = e / kRows, row = row0 + r, t = token0 + n;
    if (row >= a.n_out || t >= a.n_tokens) continue;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < kWarpsInt4; ++k) v += sums[(k * 8 * NT + n) * kPitch + r];
    if (a.base) v += to_f32(static_cast<const YT*>(a.base)[(int64_t)t * a.bs + row]);
    static_cast<YT*>(a.y)[(int64_t)t * a.ys + row] = from_f32<YT>(v);
  }
}

// y = base, or 0 (no columns).
template <typename YT>
__global__ void int4_copy(Int4Args a) {
  const int64_t n = (int64_t)a.n_tokens * a.n_out;
  for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < n; e += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = e / a.n_out, o = e - t * a.n_out;
    static_cast<YT*>(a.y)[t * a.ys + o] = a.base ? static_cast<const YT*>(a.base)[t * a.bs + o] : from_f32<YT>(0.f);
  }
}

template <typename T, typename YT, int NT, int SEG>
spmv_status launch_int4(const Int4Args& a, cudaStream_t st) {
  constexpr int MT = 2;
  const bool aligned = aligned_to(a.w, 16) && (a.n_out == 1 || a.ws % 16 == 0);
  void (*fn)(Int4Args) = aligned ? &int4_rows<T, YT, MT, NT, SEG, true> : &int4_rows<T, YT, MT, NT, SEG, false>;
  const size_t ring = (size_t)kWarpsInt4 * kRing * 16 * MT * kStepBytes;
  const size_t sums = (size_t)kWarpsInt4 * 8 * NT * (16 * MT + 1) * 4;
  const size_t smem = ring > sums ? ring : sums;
  if (!allow_smem(reinterpret_cast<const void*>(fn), smem)) return SPMV_ERR_CUDA;
  const dim3 grid((unsigned)((a.n_out + 16 * MT - 1) / (16 * MT)), (unsigned)((a.n_tokens + 8 * NT - 1) / (8 * NT)));
  return launch(fn, grid, kWarpsInt4 * 32, smem, st, a);
}

template <typename T, typename YT, int NT>
spmv_status launch_groups(const Int4Args& a, cudaStream_t st) {
  if (a.group_shift >= 7) return launch_int4<T, YT, NT, 128>(a, st);
  return a.group_shift == 6 ? launch_int4<T, YT, NT, 64>(a, st) : launch_int4<T, YT, NT, 32>(a, st);
}

template <typename T, typename YT>
spmv_status run_int4(const Int4Args& a, cudaStream_t st) {
  if (a.n_in == 0) {
    if (a.base == a.y) return SPMV_OK;
    const int64_t blocks = ((int64_t)a.n_tokens * a.n_out + 255) / 256;
    return launch(int4_copy<YT>, dim3((unsigned)(blocks < 1216 ? blocks : 1216)), 256, 0, st, a);
  }
  if (a.n_tokens <= 8) return launch_groups<T, YT, 1>(a, st);
  if (a.n_tokens <= 16) return launch_groups<T, YT, 2>(a, st);
  return a.n_tokens <= 32 ? launch_groups<T, YT, 4>(a, st) : launch_groups<T, YT, 8>(a, st);
}

}  // namespace
}  // namespace spmv

using namespace spmv;

extern "C" spmv_status spmv_int4_run(int32_t n_tokens, int32_t n_in, int32_t n_out, int32_t group,
                                     spmv_dtype dtype, const void* x, int64_t x_stride, const uint8_t* weights,
                                     int64_t weights_stride, const void* scales, spmv_dtype scales_dtype,
                                     const uint8_t* zeros, const void* base, int64_t base_stride, void* y,
                                     spmv_dtype y_dtype, int64_t y_stride, void* stream) {
  if (n_tokens < 0 || n_in < 0 || n_out < 0 || group < 1 || !op_dtype(dtype) || !op_dtype(scales_dtype) ||
      !op_dtype(y_dtype))
    return SPMV_ERR_INVALID_ARG;
  if (dtype == SPMV_F32 || (y_dtype != SPMV_F32 && y_dtype != dtype) ||
      (scales_dtype != SPMV_F32 && scales_dtype != dtype))
    return SPMV_ERR_UNSUPPORTED;
  const bool power = group >= 32 && (group & (group - 1)) == 0;
  if (!power && group < n_in) return SPMV_ERR_UNSUPPORTED;
  if (n_tokens > (1 << 18) || n_in > (1 << 30) || n_out > (1 << 30)) return SPMV_ERR_TOO_LARGE;
  const int64_t ysz = op_dtype_size(y_dtype), row_bytes = (n_in + 1ll) / 2;
  const int64_t groups = n_in == 0 ? 0 : (n_in + (int64_t)group - 1) / group;
  if (!matrix_ok(x, n_tokens, n_in, x_stride, 2, false) ||
      !matrix_ok(weights, n_out, row_bytes, weights_stride, 1, false) ||
      (base && !matrix_ok(base, n_tokens, n_out, base_stride, ysz, false)) ||
      !matrix_ok(y, n_tokens, n_out, y_stride, ysz, true) || (n_out > 0 && groups > 0 && !scales) ||
      !aligned_to(scales, op_dtype_size(scales_dtype)))
    return SPMV_ERR_INVALID_ARG;
  if (n_tokens == 0 || n_out == 0) return SPMV_OK;
  const bool in_place = base == y && (base_stride == y_stride || n_tokens == 1);
  const auto meets_y = [&](const void* p, int64_t rows, int64_t cols, int64_t stride, int64_t size) {
    return spans_overlap(p, rows, cols, stride, size, y, n_tokens, n_out, y_stride, ysz);
  };
  if ((!in_place && meets_y(base, n_tokens, n_out, base_stride, ysz)) || meets_y(x, n_tokens, n_in, x_stride, 2) ||
      meets_y(weights, n_out, row_bytes, weights_stride, 1) ||
      meets_y(scales, 1, n_out * groups, n_out * groups, op_dtype_size(scales_dtype)) ||
      meets_y(zeros, 1, n_out * groups, n_out * groups, 1))
    return SPMV_ERR_INVALID_ARG;
  Int4Args a{};
  a.n_tokens = n_tokens, a.n_in = n_in, a.n_out = n_out, a.group = group, a.groups = (int)groups;
  a.x = x, a.xs = x_stride, a.w = weights, a.ws = weights_stride;
  a.scales = scales, a.zeros = zeros, a.base = base, a.bs = base_stride, a.y = y, a.ys = y_stride;
  a.scales_f32 = scales_dtype == SPMV_F32;
  a.group_shift = 31;  // (one group)
  if (group < n_in)
    for (a.group_shift = 5; (1 << a.group_shift) < group;) ++a.group_shift;
  a.vec_x = rows_aligned(x, n_tokens, x_stride, 2, 8);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (dtype == SPMV_F16)
    return y_dtype == SPMV_F32 ? run_int4<__half, float>(a, st) : run_int4<__half, __half>(a, st);
  return y_dtype == SPMV_F32 ? run_int4<__nv_bfloat16, float>(a, st)
                             : run_int4<__nv_bfloat16, __nv_bfloat16>(a, st);
}
