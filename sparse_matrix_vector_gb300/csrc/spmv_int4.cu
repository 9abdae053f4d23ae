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
#include <cooperative_groups.h>

#include <climits>
#include <type_traits>

#include "spmv_device.cuh"
#include "spmv_types.cuh"

namespace spmv {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxWarps = 16;
constexpr int kRows = 32;              // of W, to a CTA
constexpr int kStep = 128;             // columns that a warp takes at a time
constexpr int kStepBytes = kStep / 2;
constexpr int kRing = 4;               // steps of weights in shared memory
constexpr int kStage = kRows * kStepBytes;

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
  int y_dtype;
  int split;        // CTAs that share a block of rows
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

// A CTA: 32 rows of W for 8 NT tokens, the columns split over its warps. SEG:
// columns whose sums are scaled together (a group, or a step of a longer one).
// FAST: rows of W and x start on 16-byte boundaries.
template <typename T, int NT, int SEG, bool FAST>
__global__ void __maxnreg__(NT == 1 ? 80 : NT == 2 ? 104 : 128) int4_rows(Int4Args a) {
  extern __shared__ __align__(16) unsigned char s_int4[];
  constexpr int kWords = SEG / 32, kSegs = kStep / SEG;
  const int me = threadIdx.x, warp = me >> 5, lane = me & 31, g = lane >> 2, q = lane & 3;
  const int warps = (int)blockDim.x >> 5;
  const int row0 = blockIdx.x * kRows, token0 = blockIdx.y * 8 * NT;
  const int row_bytes = (a.n_in + 1) / 2;
  const int steps = (a.n_in + kStep - 1) / kStep, whole = a.n_in / kStep;
  const int begin = (int)((int64_t)steps * warp / warps), end = (int)((int64_t)steps * (warp + 1) / warps);
  unsigned char* ring = s_int4 + warp * kRing * kStage;
  // rows g + 8 r of the CTA's, those past the end repeating the last
  int row[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) row[r] = min(g + 8 * r, a.n_out - 1 - row0);

  // this lane's pieces of a step: rows row[k], 16 bytes from column 32 q on
  const uint8_t* src = a.w + (int64_t)row0 * a.ws + q * 16;
  const uint8_t* src_row[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) src_row[r] = src + row[r] * a.ws;
  const uint32_t dst0 = smem_u32(ring) + piece_at(g, q);  // (piece_at(g + 8 r, q): 8 rows of 64 bytes on)
  const auto fetch = [&](int step) {
    if (step < end) {
      const int at = step * kStepBytes;
      const uint32_t to = (step & (kRing - 1)) * kStage;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (FAST) {
          if (step < whole) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst0 + r * 8 * kStepBytes + to),
                         "l"(src_row[r] + at)
                         : "memory");
          } else {
            const int bytes = max(0, min(16, row_bytes - at - q * 16));
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst0 + r * 8 * kStepBytes + to),
                         "l"(src_row[r] + (bytes > 0 ? at : 0)), "r"(bytes)
                         : "memory");
          }
        } else {
          const uint4 v = load_piece(src_row[r] + at, row_bytes - at - q * 16);
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst0 + r * 8 * kStepBytes + to), "r"(v.x), "r"(v.y),
                       "r"(v.z), "r"(v.w)
                       : "memory");
        }
      }
    }
    if constexpr (FAST) copy_commit();
  };

  const T* x[NT];
  bool has[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = token0 + 8 * n + g;
    has[n] = t < a.n_tokens;
    x[n] = static_cast<const T*>(a.x) + (has[n] ? (int64_t)t * a.xs : 0) + q * 8 * kWords;
  }
  // scales and zero points of rows row[r], a segment ahead
  const int64_t first_scale = (int64_t)row0 * a.groups;
  int scale_row[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) scale_row[r] = row[r] * a.groups;
  float scale[4];
  uint32_t zero[4];
  const auto load_scales = [&](int col) {
    const int k = min(col >> a.group_shift, a.groups - 1);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      scale[r] = a.scales_f32 ? __ldg(static_cast<const float*>(a.scales) + first_scale + scale_row[r] + k)
                              : to_f32(static_cast<const T*>(a.scales)[first_scale + scale_row[r] + k]);
      zero[r] = a.zeros ? __ldg(a.zeros + first_scale + scale_row[r] + k) & 15u : 8u;
    }
  };

  float acc[2][NT][4] = {};
#pragma unroll
  for (int k = 0; k < kRing - 1; ++k) fetch(begin + k);
  if (begin < end) load_scales(begin * kStep);
  for (int step = begin; step < end; ++step) {
    if constexpr (FAST) copy_wait<kRing - 2>();
    __syncwarp();
    const unsigned char* stage = ring + (step & (kRing - 1)) * kStage;
    fetch(step + kRing - 1);
#pragma unroll
    for (int seg = 0; seg < kSegs; ++seg) {
      const int col0 = step * kStep + seg * SEG;
      float s_now[4];
      Unpack<T> un[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        s_now[r] = scale[r];
        un[r].set(zero[r]);
      }
      load_scales(col0 + SEG);  // (behind the last column: the last group's again)
      // x of this lane's words: columns col0 + q * 8 kWords + 8 w
      uint4 v[NT][kWords];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
          if (FAST && step < whole) {
            v[n][k] = make_uint4(0, 0, 0, 0);
            if (has[n]) v[n][k] = __ldg(reinterpret_cast<const uint4*>(x[n] + col0 + 8 * k));
          } else {
            v[n][k] = load_x(x[n] + col0 + 8 * k, has[n] ? a.n_in - col0 - q * 8 * kWords - 8 * k : 0, FAST);
          }
        }
      // its words of the rows
      uint32_t w[4][kWords];
      const int byte = seg * (SEG / 2) + q * 4 * kWords;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const unsigned char* at = stage + piece_at(g, byte >> 4) + 8 * r * kStepBytes + (byte & 15);
        if constexpr (kWords == 4) {
          const uint4 u = *reinterpret_cast<const uint4*>(at);
          w[r][0] = u.x, w[r][1] = u.y, w[r][2] = u.z, w[r][3] = u.w;
        } else if constexpr (kWords == 2) {
          const uint2 u = *reinterpret_cast<const uint2*>(at);
          w[r][0] = u.x, w[r][1] = u.y;
        } else {
          w[r][0] = *reinterpret_cast<const uint32_t*>(at);
        }
      }
      float part[2][NT][4] = {};
#pragma unroll
      for (int k = 0; k < kWords; ++k) {
        uint32_t b[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          b[n][0] = __byte_perm(v[n][k].x, v[n][k].z, 0x5410);
          b[n][1] = __byte_perm(v[n][k].x, v[n][k].z, 0x7632);
          b[n][2] = __byte_perm(v[n][k].y, v[n][k].w, 0x5410);
          b[n][3] = __byte_perm(v[n][k].y, v[n][k].w, 0x7632);
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {
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
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[m][n][k] += s_now[2 * m + (k >> 1)] * part[m][n][k];
    }
    __syncwarp();  // (all lanes are done with the stage before it is filled again)
  }
  if constexpr (FAST) copy_wait<0>();
  __syncthreads();

  // the warps' sums, joined in their order
  constexpr int kPitch = kRows + 1;
  float* sums = reinterpret_cast<float*>(s_int4);
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        sums[(warp * 8 * NT + 8 * n + 2 * q + (k & 1)) * kPitch + 16 * m + 8 * (k >> 1) + g] = acc[m][n][k];
  __syncthreads();
  for (int e = me; e < kRows * 8 * NT; e += (int)blockDim.x) {
    const int r = e % kRows, n = e / kRows, t = token0 + n;
    if (row0 + r >= a.n_out || t >= a.n_tokens) continue;
    float v = 0.f;
    for (int k = 0; k < warps; ++k) v += sums[(k * 8 * NT + n) * kPitch + r];
    if (a.base) v += load_as_f32(a.base, a.y_dtype, (int64_t)t * a.bs + row0 + r);
    store_from_f32(a.y, a.y_dtype, (int64_t)t * a.ys + row0 + r, v);
  }
}

// ------------------------------------------------------- tensor-core tiles
// Rows at 16-byte boundaries: 256 rows of W and up to 64 tokens to a CTA, one
// CTA to an SM, on the fifth-generation tensor cores. A tile of 128 rows is
// the instruction's A operand and lives in tensor memory (a thread of the
// tile's four warps unpacks its row's columns into its own lane there), x is
// the B operand in shared memory, and the sums of a group come back from
// tensor memory to be scaled into fp32 registers. Three kinds of warps work
// at the same time: eight unpack and add up (two tiles), two bring x into the
// layout of the operand, one thread issues the instructions. The columns are
// split over a cluster's CTAs, whose sums meet in distributed shared memory.

constexpr int kTileRows = 256;
constexpr int kRowWarps = kTileRows / 32, kXWarps = 2;
constexpr int kTileThreads = (kRowWarps + kXWarps + 1) * 32;
constexpr int kRingBytes = 12 * 1024;  // of a warp's weights
constexpr int kXStages = 4;
constexpr int kMaxSplit = 8;

__device__ __forceinline__ void tmem_alloc(uint32_t* to, int columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(to)), "r"(columns)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t at, int columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns));
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(at),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_load16(uint32_t at, float (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7]), "=f"(r[8]),
        "=f"(r[9]), "=f"(r[10]), "=f"(r[11]), "=f"(r[12]), "=f"(r[13]), "=f"(r[14]), "=f"(r[15])
      : "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_store() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_load() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// D (tensor memory) = or += A (tensor memory) x B (shared memory), one instruction of 16 columns
__device__ __forceinline__ void tile_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t kind, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(kind), "r"(add)
      : "memory");
}
// The barrier hears of it when all of this thread's instructions so far are done.
__device__ __forceinline__ void tile_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
               : "memory");
}

struct TileBars {
  uint64_t x_full[kXStages], x_empty[kXStages];
  uint64_t a_full[2][2], done[2][2];  // [tile][buffer]
  uint64_t last;
  uint32_t tmem;
  int failed;
};

// Waits end: after the limit, or once another one has given up (the outputs
// are then NaN).
__device__ __forceinline__ void wait_for(uint64_t* bar, uint32_t parity, volatile int* failed) {
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    if (mbar_try_wait(bar, parity)) return;
    if ((i & 255) == 255 && *failed) return;
  }
  *failed = 1;
}

template <typename T, int N, int SEG>
__global__ void __launch_bounds__(kTileThreads, 1) int4_tiles(Int4Args a) {
  constexpr int kPieces = SEG / 32;                // 16-byte pieces of a row's step
  constexpr int kStageBytes = 32 * kPieces * 16;   // of a warp
  constexpr int kDepth = kRingBytes / kStageBytes;
  constexpr int kLine = SEG >= 64 ? 128 : 64;      // bytes of a row of the B operand: its swizzle
  constexpr int kXBytes = N * SEG * 2;
  constexpr int kAColumns = SEG / 2;               // tensor memory columns of a buffer of A
  constexpr int kColumns = 4 * kAColumns + 4 * N <= 128 ? 128 : 4 * kAColumns + 4 * N <= 256 ? 256 : 512;
  extern __shared__ __align__(1024) unsigned char s_raw[];
  __shared__ TileBars bars;
  // (the operand's swizzle goes by the address: rows of 1024-byte groups)
  unsigned char* s_tiles = s_raw + ((1024u - (smem_u32(s_raw) & 1023u)) & 1023u);
  unsigned char* x_ring = s_tiles;
  unsigned char* w_ring = s_tiles + kXStages * kXBytes;
  const int me = threadIdx.x, warp = me >> 5, lane = me & 31;
  const int rank = (int)(blockIdx.x % (unsigned)a.split), row0 = (int)(blockIdx.x / (unsigned)a.split) * kTileRows;
  const int token0 = blockIdx.y * N;
  const int steps = (a.n_in + SEG - 1) / SEG;
  const int begin = (int)((int64_t)steps * rank / a.split);
  const int count = (int)((int64_t)steps * (rank + 1) / a.split) - begin;

  if (me == 0) {
    for (int k = 0; k < kXStages; ++k) mbar_init(&bars.x_full[k], kXWarps * 32), mbar_init(&bars.x_empty[k], 1);
    for (int k = 0; k < 4; ++k) mbar_init(&bars.a_full[k >> 1][k & 1], 4), mbar_init(&bars.done[k >> 1][k & 1], 1);
    mbar_init(&bars.last, 1);
    bars.failed = 0;
    fence_mbar_init();
  }
  if (warp == kRowWarps + kXWarps) tmem_alloc(&bars.tmem, kColumns);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = bars.tmem;
  volatile int* failed = &bars.failed;

  float acc[N];
#pragma unroll
  for (int n = 0; n < N; ++n) acc[n] = 0.f;
  if (warp < kRowWarps) {
    const int tile = warp >> 2, first = row0 + 32 * warp;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // lane 32 (warp % 4) of tensor memory
    const uint32_t a_at = tmem + lanes + tile * 2 * kAColumns;
    const uint32_t d_at = tmem + lanes + 4 * kAColumns + tile * 2 * N;
    // copies: piece lane % kPieces of row k 32 / kPieces + lane / kPieces
    const int row_bytes = (a.n_in + 1) / 2, whole = a.n_in / SEG;
    const uint8_t* src[kPieces];
    uint32_t dst[kPieces];
    const uint32_t ring = smem_u32(w_ring) + warp * kRingBytes;
    const auto place = [&](int r, int p) { return (uint32_t)((r * kPieces + (p ^ ((r * kPieces >> 3) & (kPieces - 1)))) * 16); };
#pragma unroll
    for (int k = 0; k < kPieces; ++k) {
      const int r = k * (32 / kPieces) + lane / kPieces, p = lane % kPieces;
      src[k] = a.w + (int64_t)min(first + r, a.n_out - 1) * a.ws + p * 16;
      dst[k] = ring + place(r, p);
    }
    const auto fetch = [&](int s) {
      if (s < count) {
        const int step = begin + s, at = step * (SEG / 2);
        const uint32_t to = (uint32_t)(s % kDepth) * kStageBytes;
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
          if (step < whole) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst[k] + to), "l"(src[k] + at) : "memory");
          } else {
            const int bytes = max(0, min(16, row_bytes - at - (lane % kPieces) * 16));
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst[k] + to),
                         "l"(bytes > 0 ? src[k] + at : a.w), "r"(bytes)
                         : "memory");
          }
        }
      }
      copy_commit();
    };
    // this thread's row
    const int64_t scale_row = (int64_t)min(first + lane, a.n_out - 1) * a.groups;
    const auto scale_of = [&](int s) {
      const int64_t k = scale_row + min((begin + s) * SEG >> a.group_shift, a.groups - 1);
      return a.scales_f32 ? __ldg(static_cast<const float*>(a.scales) + k) : to_f32(static_cast<const T*>(a.scales)[k]);
    };
    const auto zero_of = [&](int s) {
      const int64_t k = scale_row + min((begin + s) * SEG >> a.group_shift, a.groups - 1);
      return a.zeros ? (uint32_t)__ldg(a.zeros + k) & 15u : 8u;
    };
    const auto add_up = [&](int s, float scale) {
      const int b = s & 1;
      wait_for(&bars.done[tile][b], (s >> 1) & 1, failed);
      tmem_fence_after();
      __syncwarp();
      constexpr int kAtOnce = N < 32 ? N : 32;
#pragma unroll
      for (int n0 = 0; n0 < N; n0 += kAtOnce) {
        float d[kAtOnce / 16][16];
#pragma unroll
        for (int k = 0; k < kAtOnce / 16; ++k) tmem_load16(d_at + b * N + n0 + 16 * k, d[k]);
        tmem_wait_load();
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) acc[n0 + k] = fmaf(scale, d[k / 16][k % 16], acc[n0 + k]);
      }
    };
#pragma unroll
    for (int k = 0; k < kDepth - 1; ++k) fetch(k);
    float before2 = 0.f, before1 = 0.f, now = 0.f, next = count > 0 ? scale_of(0) : 0.f;
    uint32_t next_zero = count > 0 ? zero_of(0) : 8u;
    for (int s = 0; s < count; ++s) {
      const int b = s & 1;
      before2 = before1, before1 = now, now = next;
      Unpack<T> un;
      un.set(next_zero);
      if (s + 1 < count) next = scale_of(s + 1), next_zero = zero_of(s + 1);
      copy_wait<kDepth - 2>();
      __syncwarp();
      fetch(s + kDepth - 1);
      if (s >= 2) add_up(s - 2, before2);
      const unsigned char* stage = w_ring + warp * kRingBytes + (s % kDepth) * kStageBytes;
#pragma unroll
      for (int p = 0; p < kPieces; ++p) {
        const uint4 v = *reinterpret_cast<const uint4*>(stage + place(lane, p));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        uint32_t r[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint32_t e[4];
          un.run(w[k], e);
#pragma unroll
          for (int j = 0; j < 4; ++j) r[4 * k + j] = e[j];
        }
        tmem_store16(a_at + b * kAColumns + 16 * p, r);
      }
      tmem_wait_store();
      tmem_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.a_full[tile][b]);
    }
    if (count >= 2) add_up(count - 2, before1);
    if (count >= 1) add_up(count - 1, now);
    copy_wait<0>();
  } else if (warp < kRowWarps + kXWarps) {
    // x into the operand's layout: rows of kLine bytes (tokens), 16-byte pieces
    // exchanged by the row's number; within a piece the order of Unpack
    constexpr int kChunks = SEG / 8, kMine = N * kChunks / (kXWarps * 32);
    const int id = me - kRowWarps * 32;
    for (int s = 0; s < count; ++s) {
      const int stage = s % kXStages;
      if (s >= kXStages) wait_for(&bars.x_empty[stage], ((s / kXStages) - 1) & 1, failed);
      constexpr int kAtOnce = kMine < 8 ? kMine : 8;
#pragma unroll
      for (int j0 = 0; j0 < kMine; j0 += kAtOnce) {
        uint4 v[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          const int c = id + (j0 + j) * kXWarps * 32, n = c / kChunks, col = (begin + s) * SEG + (c % kChunks) * 8;
          const T* from = static_cast<const T*>(a.x) + (int64_t)(token0 + n) * a.xs + col;
          v[j] = load_x(from, token0 + n < a.n_tokens ? a.n_in - col : 0, true);
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          const int c = id + (j0 + j) * kXWarps * 32, n = c / kChunks, kc = c % kChunks;
          uint32_t at = (uint32_t)(n * kLine + (kc % (kLine / 16)) * 16);
          at ^= (at >> 3) & (kLine == 128 ? 0x70u : 0x30u);
          at += (uint32_t)(kc / (kLine / 16)) * (N * kLine);
          *reinterpret_cast<uint4*>(x_ring + stage * kXBytes + at) =
              make_uint4(__byte_perm(v[j].x, v[j].z, 0x5410), __byte_perm(v[j].x, v[j].z, 0x7632),
                         __byte_perm(v[j].y, v[j].w, 0x5410), __byte_perm(v[j].y, v[j].w, 0x7632));
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(&bars.x_full[stage]);
    }
  } else {
    if (lane == 0) {
      // fp32 sums; both operands of T, with columns along the rows; N tokens, 128 rows
      const uint32_t type = std::is_same<T, __half>::value ? 0u : 1u;
      const uint32_t kind = 1u << 4 | type << 7 | type << 10 | (uint32_t)(N / 8) << 17 | 8u << 24;
      // rows of kLine bytes in groups of eight; bits 46-47: version, 61-63: swizzle
      const uint64_t base = (uint64_t)(8 * kLine >> 4) << 32 | 1ull << 46 | (uint64_t)(kLine == 128 ? 2 : 4) << 61 | 1ull << 16;
      for (int s = 0; s < count; ++s) {
        const int b = s & 1, stage = s % kXStages;
        wait_for(&bars.x_full[stage], (s / kXStages) & 1, failed);
        const uint32_t x_at = smem_u32(x_ring + stage * kXBytes);
#pragma unroll
        for (int tile = 0; tile < 2; ++tile) {
          wait_for(&bars.a_full[tile][b], (s >> 1) & 1, failed);
          tmem_fence_after();
          const uint32_t d = tmem + 4 * kAColumns + (tile * 2 + b) * N, op = tmem + (tile * 2 + b) * kAColumns;
#pragma unroll
          for (int k = 0; k < SEG / 16; ++k) {
            const uint32_t at = x_at + (k * 32 / kLine) * (N * kLine) + k * 32 % kLine;
            tile_mma(d, op + 8 * k, base | (uint64_t)((at >> 4) & 0x3fff), kind, k > 0);
          }
          tile_commit(&bars.done[tile][b]);
        }
        tile_commit(&bars.x_empty[stage]);
      }
      tile_commit(&bars.last);
      if (!mbar_wait_bounded(&bars.last, 0)) *failed = 1;  // (tensor memory is given back behind it)
    }
    __syncwarp();
  }

  // The sums: [token][row] in shared memory, then the cluster's, in order.
  __syncthreads();
  float* sums = reinterpret_cast<float*>(s_tiles);
  if (warp < kRowWarps) {
#pragma unroll
    for (int n = 0; n < N; ++n) sums[n * kTileRows + 32 * warp + lane] = acc[n];
  }
  tmem_fence_before();
  cg::cluster_group cluster = cg::this_cluster();
  if (a.split > 1)
    cluster.sync();
  else
    __syncthreads();
  if (warp == kRowWarps + kXWarps) {
    tmem_fence_after();
    tmem_free(tmem, kColumns);
  }
  const int lo = kTileRows * rank / a.split, rows = kTileRows * (rank + 1) / a.split - lo;
  const int tokens = min(N, a.n_tokens - token0);
  for (int e = me; e < rows * tokens; e += kTileThreads) {
    const int n = e / rows, r = lo + e % rows;
    if (row0 + r >= a.n_out) continue;
    float v = 0.f;
    for (int k = 0; k < a.split; ++k)
      v += (a.split > 1 ? cluster.map_shared_rank(sums, k) : sums)[n * kTileRows + r];
    if (*failed) v = NAN;
    if (a.base) v += load_as_f32(a.base, a.y_dtype, (int64_t)(token0 + n) * a.bs + row0 + r);
    store_from_f32(a.y, a.y_dtype, (int64_t)(token0 + n) * a.ys + row0 + r, v);
  }
  if (a.split > 1) cluster.sync();  // (the others read this CTA's sums)
}

// y = base, or 0 (no columns).
__global__ void int4_copy(Int4Args a) {
  const int64_t n = (int64_t)a.n_tokens * a.n_out;
  for (int64_t e = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; e < n; e += (int64_t)gridDim.x * blockDim.x) {
    const int64_t t = e / a.n_out, o = e - t * a.n_out;
    const float v = a.base ? load_as_f32(a.base, a.y_dtype, t * a.bs + o) : 0.f;
    store_from_f32(a.y, a.y_dtype, t * a.ys + o, v);
  }
}

template <typename T, int NT, int SEG>
spmv_status launch_rows(const Int4Args& a, cudaStream_t st) {
  const bool fast = aligned_to(a.w, 16) && (a.n_out <= 1 || a.ws % 16 == 0) && a.vec_x;
  void (*fn)(Int4Args) = fast ? &int4_rows<T, NT, SEG, true> : &int4_rows<T, NT, SEG, false>;
  const int64_t blocks = (a.n_out + kRows - 1ll) / kRows, groups = (a.n_tokens + 8ll * NT - 1) / (8 * NT);
  // as many warps to a CTA as one wave of 24 warps per SM has for it
  int warps = 4;
  while (warps < kMaxWarps && blocks * groups * warps * 2 <= 24 * 152) warps *= 2;
  const size_t ring = (size_t)warps * kRing * kStage;
  const size_t sums = (size_t)warps * 8 * NT * (kRows + 1) * 4;
  const size_t smem = ring > sums ? ring : sums;
  if (!allow_smem(reinterpret_cast<const void*>(fn), smem)) return SPMV_ERR_CUDA;
  return launch(fn, dim3((unsigned)blocks, (unsigned)groups), warps * 32, smem, st, a);
}

template <typename T, int N, int SEG>
spmv_status launch_tiles(Int4Args a, cudaStream_t st) {
  const void* fn = reinterpret_cast<const void*>(&int4_tiles<T, N, SEG>);
  const size_t rings = (size_t)kXStages * N * SEG * 2 + (size_t)kRowWarps * kRingBytes;
  const size_t sums = (size_t)N * kTileRows * 4;
  // (more than half of an SM's: two CTAs there would share its tensor memory)
  size_t smem = (rings > sums ? rings : sums) + 1024;
  if (smem < 120 * 1024) smem = 120 * 1024;
  if (!allow_smem(fn, smem)) return SPMV_ERR_CUDA;
  const int64_t blocks = (a.n_out + kTileRows - 1ll) / kTileRows, groups = (a.n_tokens + N - 1ll) / N;
  // the columns over as many CTAs as the device holds together
  a.split = kMaxSplit;
  while (a.split > 1 && (blocks * groups * a.split > 152 ||
                         resident_clusters(fn, a.split, kTileThreads, smem) < blocks * groups))
    --a.split;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks * a.split), (unsigned)groups);
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.split;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {&a};
  return status_of(cudaLaunchKernelExC(&cfg, fn, args));
}

template <typename T, int N>
spmv_status tile_groups(const Int4Args& a, cudaStream_t st) {
  if (a.group_shift >= 7) return launch_tiles<T, N, 128>(a, st);
  return a.group_shift == 6 ? launch_tiles<T, N, 64>(a, st) : launch_tiles<T, N, 32>(a, st);
}

template <typename T, int NT>
spmv_status launch_groups(const Int4Args& a, cudaStream_t st) {
  if (a.group_shift >= 7) return launch_rows<T, NT, 128>(a, st);
  return a.group_shift == 6 ? launch_rows<T, NT, 64>(a, st) : launch_rows<T, NT, 32>(a, st);
}

template <typename T>
spmv_status run_int4(const Int4Args& a, cudaStream_t st) {
  if (a.n_in == 0) {
    if (a.base == a.y) return SPMV_OK;
    const int64_t blocks = ((int64_t)a.n_tokens * a.n_out + 255) / 256;
    return launch(int4_copy, dim3((unsigned)(blocks < 1216 ? blocks : 1216)), 256, 0, st, a);
  }
  const bool fast = aligned_to(a.w, 16) && (a.n_out <= 1 || a.ws % 16 == 0) && a.vec_x;
  if (fast) {
    if (a.n_tokens <= 16) return tile_groups<T, 16>(a, st);
    return a.n_tokens <= 32 ? tile_groups<T, 32>(a, st) : tile_groups<T, 64>(a, st);
  }
  if (a.n_tokens <= 8) return launch_groups<T, 1>(a, st);
  return a.n_tokens <= 16 ? launch_groups<T, 2>(a, st) : launch_groups<T, 4>(a, st);
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
  a.y_dtype = y_dtype;
  a.scales_f32 = scales_dtype == SPMV_F32;
  a.group_shift = 31;  // (one group)
  if (group < n_in)
    for (a.group_shift = 5; (1 << a.group_shift) < group;) ++a.group_shift;
  a.vec_x = rows_aligned(x, n_tokens, x_stride, 2, 8);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == SPMV_F16 ? run_int4<__half>(a, st) : run_int4<__nv_bfloat16>(a, st);
}
