// Layer norm of rows and its gradient (spmv_layernorm,
// spmv_layernorm_backward).
//
//   mean = sum x / n, rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
//   y = (x - mean) rstd w + b
//   g = dy w, c = x - mean:
//   dx = rstd g - rstd mean(g) - c rstd^3 mean(g c)
//   dw = sum over rows of dy c rstd, db = sum over rows of dy
//
// Both are bound by moving the rows: some ten operations per element, each
// read once and written once. All arithmetic is fp32; a value is rounded once,
// to the type of the tensor it goes to. Measured, in us, and as a share of the
// 6.79 TB/s of a plain copy:
//   norm      8192 x 12288 fp32 -> fp16  89 (1.00)   16384 x 4096  62 (0.96)
//             8192 x 12288 bf16          74 (0.80)   16384 x 4096  45 (0.87)
//   gradient  8192 x 12288 fp32, fp16   166 (0.89)   16384 x 4096 106 (0.93)
//             8192 x 12288 bf16         120 (0.74)   16384 x 4096  81 (0.73)
// In 16 bits the gradient is bound by its instructions, some 14 per element
// (unpacking x and dy twice, once for the sums and once for dx).
// Unaligned rows move element by element: 8192 x 5003 bf16 64 us (0.38), its
// gradient 94 (0.39); 1023 x 5003 12.4 us, of which a launch is 4.3.
#include <climits>
#include <type_traits>

#include "spmv_device.cuh"
#include "spmv_types.cuh"

namespace spmv {
namespace {

// Sum over the CTA, in every thread, in a fixed order. One barrier; s_red
// (32 floats) must not be in use by an earlier call when this one starts.
__device__ __forceinline__ float cta_sum_all(float v, float* s_red) {
  v = warp_sum(v);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) s_red[warp] = v;
  __syncthreads();
  return warp_sum(lane < (int)(blockDim.x >> 5) ? s_red[lane] : 0.f);
}

// Columns a thread holds of its rows, and the threads a CTA has at most with
// them: more columns, or the addresses of single elements, take more
// registers and leave room for fewer threads.
constexpr int most_threads(int cols, bool aligned) {
  return cols == 8 ? 640 : cols == 16 && aligned ? 768 : 512;
}

template <typename XT, typename YT>
struct ForwardArgs {
  int64_t n_rows;
  int n_cols;
  const XT* x;
  int64_t xs;
  const void *w, *b;
  int pt;
  float eps;
  YT* y;
  int64_t ys;
  float *mean, *rstd;
};

// Forward, one pass over x: a group of threads (a warp, or the CTA) takes
// rows in turn, each thread the same CPT columns of every row, whose weight
// and bias it keeps in registers. STAGES - 1 rows are on their way into
// shared memory while one is worked on. STAGES 0: rows that are not 16-byte
// aligned, loaded directly, the next one asked from L2 a row ahead; weight and
// bias are in shared memory then, which leaves registers for more CTAs. Mean and
// variance are taken one after the other, the variance from the centred
// values: no cancellation. The arithmetic is on pairs (fp32x2 instructions).
template <typename XT, typename YT, int VEC, int CPT, int STAGES, bool WARP>
__global__ void __launch_bounds__(WARP ? kThreads : most_threads(CPT, STAGES > 0),
                                  STAGES == 0 && CPT <= 16 ? 2 : 1)
layernorm_fused(ForwardArgs<XT, YT> p) {
  constexpr int NV = CPT / VEC;
  constexpr bool kAligned = STAGES > 0;
  using PX = Pack<XT, VEC>;
  extern __shared__ __align__(16) unsigned char s_dyn[];
  __shared__ float s_red[2][32];
  const Cols<VEC, kAligned> cols{WARP ? (int)threadIdx.x & 31 : (int)threadIdx.x,
                                 WARP ? 32 : (int)blockDim.x, p.n_cols};
  const int64_t step = (int64_t)gridDim.x * (WARP ? kWarps : 1);
  const int64_t first = (int64_t)blockIdx.x * (WARP ? kWarps : 1) + (WARP ? threadIdx.x >> 5 : 0);
  const float inv = 1.f / (float)p.n_cols;
  // ring of stages, vector i of thread t at [stage][i][t]
  PX* ring = reinterpret_cast<PX*>(s_dyn);
  const auto slot = [&](int stage, int i) {
    return (stage * NV + i) * (int)blockDim.x + (int)threadIdx.x;
  };
  const auto fetch = [&](int64_t r, int stage) {
    if (r < p.n_rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (cols.has(i))
          copy_async<sizeof(PX)>(&ring[slot(stage, i)], p.x + r * p.xs + cols.col(i, 0));
    }
    copy_commit();
  };
  if constexpr (STAGES > 0) {
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) fetch(first + k * step, k);
  }
  // unaligned rows: pair j of thread t at [weight, bias][j][t]
  float2* s_param = reinterpret_cast<float2*>(s_dyn) + threadIdx.x;
  float2 g[NV][VEC / 2], o[NV][VEC / 2];
  cols.load_param(p.w, p.pt, 1.f, g);
  if constexpr (STAGES == 0) {
#pragma unroll
    for (int j = 0; j < CPT / 2; ++j) s_param[j * blockDim.x] = g[j / (VEC / 2)][j % (VEC / 2)];
  }
  cols.load_param(p.b, p.pt, 0.f, o);
  if constexpr (STAGES == 0) {
#pragma unroll
    for (int j = 0; j < CPT / 2; ++j)
      s_param[(CPT / 2 + j) * blockDim.x] = o[j / (VEC / 2)][j % (VEC / 2)];
  }
  int stage = 0;
  for (int64_t r = first; r < p.n_rows; r += step) {
    PX in[NV];
    if constexpr (STAGES > 0) {
      // the stage before this one is free: this thread read it a row ago
      fetch(r + (STAGES - 1) * step, stage == 0 ? STAGES - 1 : stage - 1);
      copy_wait<STAGES - 1>();
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (cols.has(i)) in[i] = ring[slot(stage, i)];
      stage = stage + 1 == STAGES ? 0 : stage + 1;
    } else {
      cols.load(p.x + r * p.xs, in, true);
      if (r + step < p.n_rows) cols.prefetch(p.x + (r + step) * p.xs);
    }
    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (cols.has(i)) {
#pragma unroll
        for (int k = 0; k < VEC / 2; ++k) {
          float2 v = pair_f32(in[i], k);
          if (!cols.has(i, 2 * k)) v.x = 0.f;
          if (!cols.has(i, 2 * k + 1)) v.y = 0.f;
          s2 = __fadd2_rn(s2, v);
        }
      }
    const float s = s2.x + s2.y;
    const float mean = (WARP ? warp_sum(s) : cta_sum_all(s, s_red[0])) * inv;
    const float2 off = make_float2(-mean, -mean);
    float2 q2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (cols.has(i)) {
#pragma unroll
        for (int k = 0; k < VEC / 2; ++k) {
          float2 c = __fadd2_rn(pair_f32(in[i], k), off);
          if (!cols.has(i, 2 * k)) c.x = 0.f;
          if (!cols.has(i, 2 * k + 1)) c.y = 0.f;
          q2 = __ffma2_rn(c, c, q2);
        }
      }
    const float q = q2.x + q2.y;
    const float rstd = rsqrtf((WARP ? warp_sum(q) : cta_sum_all(q, s_red[1])) * inv + p.eps);
    const float2 scale = make_float2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (cols.has(i)) {
        Pack<YT, VEC> out;
#pragma unroll
        for (int k = 0; k < VEC / 2; ++k) {
          const float2 c = __fadd2_rn(pair_f32(in[i], k), off);
          const int j = i * (VEC / 2) + k;
          const float2 gk = STAGES == 0 ? s_param[j * blockDim.x] : g[i][k];
          const float2 ok = STAGES == 0 ? s_param[(CPT / 2 + j) * blockDim.x] : o[i][k];
          set_pair(out, k, __ffma2_rn(__fmul2_rn(c, scale), gk, ok));
        }
        cols.store(p.y + r * p.ys, i, out);
      }
    if (cols.me == 0) {
      if (p.mean) p.mean[r] = mean;
      if (p.rstd) p.rstd[r] = rstd;
    }
  }
}

// Forward, rows too long for registers: one row per CTA step, three passes
// over it (mean, variance, output), the second and third mostly from L2.
template <typename XT, typename YT>
__global__ void __launch_bounds__(kThreads)
layernorm_rows(ForwardArgs<XT, YT> p) {
  __shared__ float s_red[2][32];
  const int n_cols = p.n_cols;
  for (int64_t r = blockIdx.x; r < p.n_rows; r += gridDim.x) {
    const XT* xr = p.x + r * p.xs;
    YT* yr = p.y + r * p.ys;
    float s = 0.f;
    for (int j = threadIdx.x; j < n_cols; j += kThreads) s += to_f32(xr[j]);
    const float mean = cta_sum_all(s, s_red[0]) / (float)n_cols;
    float q = 0.f;
    for (int j = threadIdx.x; j < n_cols; j += kThreads) {
      const float c = to_f32(xr[j]) - mean;
      q += c * c;
    }
    const float rstd = rsqrtf(cta_sum_all(q, s_red[1]) / (float)n_cols + p.eps);
    for (int j = threadIdx.x; j < n_cols; j += kThreads) {
      const float g = p.w ? load_as_f32(p.w, p.pt, j) : 1.f;
      const float o = p.b ? load_as_f32(p.b, p.pt, j) : 0.f;
      yr[j] = from_f32<YT>((to_f32(xr[j]) - mean) * rstd * g + o);
    }
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[r] = mean;
      if (p.rstd) p.rstd[r] = rstd;
    }
  }
}

template <typename XT, typename YT>
struct BackwardArgs {
  int64_t n_rows;
  int n_cols;
  const YT* dy;
  int64_t dys;
  const XT* x;
  int64_t xs;
  const void* w;
  int pt;
  const float *mean, *rstd;
  XT* dx;        // or null
  int64_t dxs;
  float* part;   // row_ctas x {dweight, dbias} x n_cols partial sums, or null
  int row_ctas;  // CTAs that take rows; the others take columns (column_sums)
  void *dweight, *dbias;  // what column_sums writes
};

// Sums of N values over the CTA, in every thread, in a fixed order. One
// barrier; s_red must not be in use by an earlier call.
template <int N>
__device__ __forceinline__ void cta_sums_all(float (&v)[N], float (*s_red)[N]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_sum(v[k]);
  if (lane == 0) {
#pragma unroll
    for (int k = 0; k < N; ++k) s_red[warp][k] = v[k];
  }
  __syncthreads();
  const bool on = lane < (int)(blockDim.x >> 5);
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = warp_sum(on ? s_red[lane][k] : 0.f);
}

// dweight and dbias of the 32 columns from c0, by one CTA, straight from x and
// dy: each warp sums every warps-th row, then the warps' sums in order. For
// calls so small that their rows are still in L2: one launch and no workspace.
template <typename XT, typename YT>
__device__ __forceinline__ void column_sums(const BackwardArgs<XT, YT>& p, int c0) {
  __shared__ float s_dw[32][32], s_db[32][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int c = c0 + lane, at = min(c, p.n_cols - 1);
  const int n = (int)p.n_rows;
  float dw = 0.f, db = 0.f;
  // 32 of the warp's rows at a time, whose statistics the lanes load
  const XT* x = p.x + at;
  const YT* dy = p.dy + at;
  for (int base = warp; base < n; base += 32 * warps) {
    const int mine = min(base + lane * warps, n - 1);
    const float m_lane = p.mean[mine], rs_lane = p.rstd[mine];
#pragma unroll 1
    for (int k0 = 0; k0 < 32 && base + k0 * warps < n; k0 += 8) {
      XT xv[8];
      YT dv[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int64_t r = min(base + (k0 + k) * warps, n - 1);
        xv[k] = x[r * p.xs];
        dv[k] = dy[r * p.dys];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float m = __shfl_sync(0xffffffffu, m_lane, k0 + k);
        const float rs = __shfl_sync(0xffffffffu, rs_lane, k0 + k);
        if (base + (k0 + k) * warps < n) {
          const float d = to_f32(dv[k]);
          dw += d * ((to_f32(xv[k]) - m) * rs);
          db += d;
        }
      }
    }
  }
  s_dw[warp][lane] = dw;
  s_db[warp][lane] = db;
  __syncthreads();
  if (warp > 0 || c >= p.n_cols) return;
  for (int k = 1; k < warps; ++k) {
    dw += s_dw[k][lane];
    db += s_db[k][lane];
  }
  if (p.dweight) store_from_f32(p.dweight, p.pt, c, dw);
  if (p.dbias) store_from_f32(p.dbias, p.pt, c, db);
}

// Backward, one pass over x and dy: a group of threads (a warp, or the CTA)
// takes ROWS rows at a time, each thread the same CPT columns of every row,
// whose weight it keeps and whose dweight and dbias it sums in registers.
// With c = x - mean, a row needs the sums of g and of g * c:
//   dx = rstd * g - rstd * mean(g) - c * rstd^3 * mean(g * c).
// STAGES - 1 sets of rows are on their way into shared memory while one is
// worked on, twice, from there. STAGES 0: rows that are not 16-byte aligned,
// held in registers, the next one asked from L2 ahead; the weight is in
// shared memory then.
template <typename XT, typename YT, int VEC, int CPT, int STAGES, int ROWS, bool WARP>
__global__ void __launch_bounds__(WARP ? kThreads : most_threads(CPT, STAGES > 0),
                                  !WARP ? 1 : CPT == 8 ? 3 : 2)
layernorm_backward_fused(BackwardArgs<XT, YT> p) {
  constexpr int NV = CPT / VEC;
  constexpr bool kAligned = STAGES > 0;
  using PX = Pack<XT, VEC>;
  using PY = Pack<YT, VEC>;
  extern __shared__ __align__(16) unsigned char s_dyn[];
  __shared__ float s_red[2][32][2 * ROWS];
  const Cols<VEC, kAligned> cols{WARP ? (int)threadIdx.x & 31 : (int)threadIdx.x,
                                 WARP ? 32 : (int)blockDim.x, p.n_cols};
  const int n = p.n_cols;
  // the CTAs for columns come first: they take longest
  const int row_cta = (int)blockIdx.x - ((int)gridDim.x - p.row_ctas);
  if (row_cta < 0) {
    column_sums(p, 32 * (int)blockIdx.x);
    return;
  }
  const int64_t step = (int64_t)p.row_ctas * (WARP ? kWarps : 1);
  const int64_t first = (int64_t)row_cta * (WARP ? kWarps : 1) + (WARP ? threadIdx.x >> 5 : 0);
  const float inv = 1.f / (float)n;
  // ring of row slots, vector i of thread t at [slot][i][t]
  PX* ring_x = reinterpret_cast<PX*>(s_dyn);
  PY* ring_y = reinterpret_cast<PY*>(s_dyn + (size_t)STAGES * ROWS * NV * blockDim.x * sizeof(PX));
  const auto place = [&](int slot, int i) {
    return (slot * NV + i) * (int)blockDim.x + (int)threadIdx.x;
  };
  const auto fetch = [&](int64_t r, int stage) {
#pragma unroll
    for (int h = 0; h < ROWS; ++h)
      if (r + h * step < p.n_rows) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (cols.has(i)) {
            const int64_t at = r + h * step;
            copy_async<sizeof(PX)>(&ring_x[place(stage * ROWS + h, i)],
                                   p.x + at * p.xs + cols.col(i, 0));
            copy_async<sizeof(PY)>(&ring_y[place(stage * ROWS + h, i)],
                                   p.dy + at * p.dys + cols.col(i, 0));
          }
      }
    copy_commit();
  };
  if constexpr (STAGES > 0) {
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) fetch(first + k * ROWS * step, k);
  }
  // unaligned rows: pair j of thread t's weight at [j][t]
  float2* s_w = reinterpret_cast<float2*>(s_dyn) + threadIdx.x;
  float2 w[NV][VEC / 2];
  cols.load_param(p.w, p.pt, 1.f, w);
  if constexpr (STAGES == 0) {
#pragma unroll
    for (int j = 0; j < CPT / 2; ++j) s_w[j * blockDim.x] = w[j / (VEC / 2)][j % (VEC / 2)];
  }
  const auto weight = [&](int i, int k) {
    return STAGES == 0 ? s_w[(i * (VEC / 2) + k) * blockDim.x] : w[i][k];
  };

  float2 dw[NV][VEC / 2], db[NV][VEC / 2];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < VEC / 2; ++k) dw[i][k] = db[i][k] = make_float2(0.f, 0.f);
  float m[ROWS], rs[ROWS], m_next[ROWS] = {}, rs_next[ROWS] = {};
#pragma unroll
  for (int h = 0; h < ROWS; ++h)
    if (first + h * step < p.n_rows)
      m_next[h] = p.mean[first + h * step], rs_next[h] = p.rstd[first + h * step];
  int stage = 0, turn = 0;
  PX x[STAGES > 0 ? 1 : NV] = {};  // unaligned rows
  PY dy[STAGES > 0 ? 1 : NV] = {};
  const auto x_of = [&](int h, int i) {  // vector i of row h of the set
    if constexpr (STAGES > 0)
      return ring_x[place(stage * ROWS + h, i)];
    else
      return x[i];
  };
  const auto dy_of = [&](int h, int i) {
    if constexpr (STAGES > 0)
      return ring_y[place(stage * ROWS + h, i)];
    else
      return dy[i];
  };
  for (int64_t r = first; r < p.n_rows; r += ROWS * step) {
#pragma unroll
    for (int h = 0; h < ROWS; ++h) {
      m[h] = m_next[h], rs[h] = rs_next[h];
      const int64_t at = r + (ROWS + h) * step;
      if (at < p.n_rows) m_next[h] = p.mean[at], rs_next[h] = p.rstd[at];
    }
    if constexpr (STAGES > 0) {
      // the stage before this one is free: this thread is done with it
      fetch(r + (STAGES - 1) * ROWS * step, stage == 0 ? STAGES - 1 : stage - 1);
      copy_wait<STAGES - 1>();
    } else {
      cols.load(p.x + r * p.xs, x, true);
      cols.load(p.dy + r * p.dys, dy, true);  // (past the end: zeros, which count nothing)
      if (r + step < p.n_rows) {
        cols.prefetch(p.x + (r + step) * p.xs);
        cols.prefetch(p.dy + (r + step) * p.dys);
      }
    }
    float sums[2 * ROWS];
#pragma unroll
    for (int h = 0; h < ROWS; ++h) {
      float2 sg = make_float2(0.f, 0.f), sgc = sg;
      if (h == 0 || r + h * step < p.n_rows) {
        const float2 off = make_float2(-m[h], -m[h]), scale = make_float2(rs[h], rs[h]);
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (cols.has(i)) {
            const PX xi = x_of(h, i);
            const PY di = dy_of(h, i);
#pragma unroll
            for (int k = 0; k < VEC / 2; ++k) {
              const float2 d = pair_f32(di, k), c = __fadd2_rn(pair_f32(xi, k), off);
              const float2 gk = __fmul2_rn(d, weight(i, k));
              sg = __fadd2_rn(sg, gk);
              sgc = __ffma2_rn(gk, c, sgc);
              dw[i][k] = __ffma2_rn(__fmul2_rn(d, scale), c, dw[i][k]);
              db[i][k] = __fadd2_rn(db[i][k], d);
            }
          }
      }
      sums[2 * h] = sg.x + sg.y;
      sums[2 * h + 1] = sgc.x + sgc.y;
    }
    if (p.dx) {
      if constexpr (WARP) {
#pragma unroll
        for (int k = 0; k < 2 * ROWS; ++k) sums[k] = warp_sum(sums[k]);
      } else {
        cta_sums_all<2 * ROWS>(sums, s_red[turn]);
        turn ^= 1;
      }
#pragma unroll
      for (int h = 0; h < ROWS; ++h) {
        if (h > 0 && r + h * step >= p.n_rows) break;
        const float2 off = make_float2(-m[h], -m[h]), scale = make_float2(rs[h], rs[h]);
        const float a = -rs[h] * (sums[2 * h] * inv);
        const float b = -rs[h] * (rs[h] * (rs[h] * (sums[2 * h + 1] * inv)));
        const float2 fa = make_float2(a, a), fb = make_float2(b, b);
#pragma unroll
        for (int i = 0; i < NV; ++i)
          if (cols.has(i)) {
            const PX xi = x_of(h, i);
            const PY di = dy_of(h, i);
            PX out;
#pragma unroll
            for (int k = 0; k < VEC / 2; ++k) {
              const float2 c = __fadd2_rn(pair_f32(xi, k), off);
              const float2 gk = __fmul2_rn(pair_f32(di, k), weight(i, k));
              set_pair(out, k, __ffma2_rn(c, fb, __ffma2_rn(gk, scale, fa)));
            }
            cols.store(p.dx + (r + h * step) * p.dxs, i, out);
          }
      }
    }
    if constexpr (STAGES > 0) stage = stage + 1 == STAGES ? 0 : stage + 1;
  }
  pdl_launch_dependents();
  if (!p.part) return;
  float* part = p.part + (int64_t)row_cta * 2 * n;
  if constexpr (WARP) {
    // the warps' sums, added up in warp order in shared memory
    copy_wait<0>();
    float* s_dw = reinterpret_cast<float*>(s_dyn);
    float* s_db = s_dw + n;
    for (int t = 0; t < kWarps; ++t) {
      __syncthreads();
      if ((int)(threadIdx.x >> 5) != t) continue;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (cols.has(i)) {
#pragma unroll
          for (int k = 0; k < VEC / 2; ++k) {
            if constexpr (kAligned) {
              float2* pw = reinterpret_cast<float2*>(s_dw + cols.col(i, 2 * k));
              float2* pb = reinterpret_cast<float2*>(s_db + cols.col(i, 2 * k));
              *pw = t ? __fadd2_rn(*pw, dw[i][k]) : dw[i][k];
              *pb = t ? __fadd2_rn(*pb, db[i][k]) : db[i][k];
            } else {
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (cols.has(i, 2 * k + e)) {
                  const int c = cols.col(i, 2 * k + e);
                  s_dw[c] = (t ? s_dw[c] : 0.f) + (e ? dw[i][k].y : dw[i][k].x);
                  s_db[c] = (t ? s_db[c] : 0.f) + (e ? db[i][k].y : db[i][k].x);
                }
            }
          }
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * n; c += kThreads) part[c] = s_dw[c];
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (cols.has(i)) {
        Pack<float, VEC> pw, pb;
#pragma unroll
        for (int k = 0; k < VEC / 2; ++k) {
          set_pair(pw, k, dw[i][k]);
          set_pair(pb, k, db[i][k]);
        }
        cols.store(part, i, pw);
        cols.store(part + n, i, pb);
      }
  }
}

// f(column, x, dy) for this thread's columns of a row, kFew loads of each
// under way at a time. (Loads past the end repeat the last column; their
// values are not used.)
constexpr int kFew = 8;

template <typename XT, typename YT, typename F>
__device__ __forceinline__ void for_row(const XT* x, const YT* dy, int n, F&& f) {
  for (int64_t j0 = threadIdx.x; j0 < n; j0 += kFew * kThreads) {
    XT xv[kFew];
    YT dv[kFew];
#pragma unroll
    for (int k = 0; k < kFew; ++k) {
      const int64_t j = min(j0 + k * kThreads, (int64_t)n - 1);
      xv[k] = x[j];
      dv[k] = dy[j];
    }
#pragma unroll
    for (int k = 0; k < kFew; ++k)
      if (j0 + k * kThreads < n) f((int)(j0 + k * kThreads), to_f32(xv[k]), to_f32(dv[k]));
  }
}

// Backward, rows too long for registers: dx, one row per CTA step.
template <typename XT, typename YT>
__global__ void __launch_bounds__(kThreads) layernorm_dx_rows(BackwardArgs<XT, YT> p) {
  __shared__ float s_red[2][32][2];
  int turn = 0;
  for (int64_t r = blockIdx.x; r < p.n_rows; r += gridDim.x) {
    const float m = p.mean[r], rs = p.rstd[r];
    const YT* dy = p.dy + r * p.dys;
    const XT* x = p.x + r * p.xs;
    float sg = 0.f, sgx = 0.f;
    for_row(x, dy, p.n_cols, [&](int j, float v, float d) {
      const float g = d * (p.w ? load_as_f32(p.w, p.pt, j) : 1.f);
      sg += g;
      sgx += g * ((v - m) * rs);
    });
    float sums[2] = {sg, sgx};
    cta_sums_all<2>(sums, s_red[turn]);
    turn ^= 1;
    sg = sums[0] / (float)p.n_cols;
    sgx = sums[1] / (float)p.n_cols;
    for_row(x, dy, p.n_cols, [&](int j, float v, float d) {
      const float g = d * (p.w ? load_as_f32(p.w, p.pt, j) : 1.f);
      p.dx[r * p.dxs + j] = from_f32<XT>(rs * (g - sg - (v - m) * rs * sgx));
    });
  }
}

// ... and dweight and dbias: partial sums of a block of rows, a thread per
// column.
constexpr int kLongParts = 64;

template <typename XT, typename YT>
__global__ void __launch_bounds__(kThreads) layernorm_params_part(BackwardArgs<XT, YT> p) {
  const int j = blockIdx.x * kThreads + threadIdx.x;
  if (j >= p.n_cols) return;
  const int64_t per = (p.n_rows + kLongParts - 1) / kLongParts;
  const int64_t lo = blockIdx.y * per, hi = lo + per < p.n_rows ? lo + per : p.n_rows;
  float dw = 0.f, db = 0.f;
#pragma unroll 8
  for (int64_t r = lo; r < hi; ++r) {
    const float d = to_f32(p.dy[r * p.dys + j]);
    dw += d * ((to_f32(p.x[r * p.xs + j]) - p.mean[r]) * p.rstd[r]);
    db += d;
  }
  p.part[(int64_t)blockIdx.y * 2 * p.n_cols + j] = dw;
  p.part[((int64_t)blockIdx.y * 2 + 1) * p.n_cols + j] = db;
}

// dweight and dbias from `parts` partial sums: 32 columns per CTA, each warp
// taking every kSumWarps-th part, then the warps' sums in order.
constexpr int kSumWarps = 16;

__global__ void __launch_bounds__(kSumWarps * 32)
layernorm_params_sum(int n_cols, int parts, const float* part, void* dw_out, void* db_out, int pt) {
  __shared__ float s_part[kSumWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;  // column of {dweight, dbias}
  pdl_wait();
  float v = 0.f;
  if (c < 2ll * n_cols) {
    const float* q = part + c;
#pragma unroll 8
    for (int k = warp; k < parts; k += kSumWarps) v += q[(int64_t)k * 2 * n_cols];
  }
  s_part[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || c >= 2ll * n_cols) return;
  v = 0.f;
#pragma unroll
  for (int k = 0; k < kSumWarps; ++k) v += s_part[k][lane];
  if (c < n_cols) {
    if (dw_out) store_from_f32(dw_out, pt, c, v);
  } else if (db_out) {
    store_from_f32(db_out, pt, c - n_cols, v);
  }
}

constexpr int kSms = 152;
constexpr size_t kSmemPerSm = 228 * 1024;
constexpr size_t kSmemStatic = 10 * 1024;  // of a backward CTA, with what the system reserves

// How the rows of a call are cut: a warp per row or a CTA per row, columns
// per thread (0: rows too long for registers), threads, CTAs. In us, with the
// other choice measured beside it:
// - A warp takes rows of up to 512 columns, without barriers: 65536 x 256 fp16
//   18 (CTAs: 35), gradient 28 (36); unaligned 65536 x 301 bf16 39 (64).
// - Longer rows take the columns per thread with which an SM holds two CTAs at
//   least: one works while the other waits for its sums. Norm in 16 bits, 32
//   columns up to 8192: 16384 x 8192 bf16 86 (16 columns: 113), x 4096 45 (50);
//   below 2048 they leave too few warps. Of fp32 the ring of 32 columns is too
//   large to gain: 16384 x 8192 134 (16 columns: 128). Gradient, 8 columns up
//   to 2048: 32768 x 1024 bf16 45 (16: 53); 32 columns from 6144 to 8192:
//   16384 x 8192 bf16 149 (16: 177).
// - Above that one CTA fills an SM: 16 columns, whose threads need fewer
//   registers, while they reach: gradient of 8192 x 12288 bf16 120 (32: 137).
// - The registers would hold more threads of 8 fp32 columns, but then the
//   rings' requests get in each other's way: gradient of 32768 x 1024 fp32 60
//   (1024 threads per SM: 72).
// - Unaligned rows, whose loads go to registers: 16 columns, gradient of
//   16384 x 4001 bf16 115 (8: 159), but 8 where 16 leave one CTA per SM: 8192 x
//   5003 92 (16: 100).
struct RowShape {
  bool warp;
  int cols, threads, grid;
};

// xs, ys: bytes of an element of x and of y (or dy).
RowShape row_shape(int64_t n_rows, int n_cols, size_t xs, size_t ys, bool aligned, bool forward) {
  RowShape s{};
  int per_sm = 0;  // CTAs that an SM's registers hold
  int64_t groups = n_rows;
  if (n_cols <= 512) {
    s.warp = true;
    s.cols = n_cols <= 256 ? 8 : 16;
    s.threads = kThreads;
    per_sm = (s.cols == 8 ? 3 : 2) + (forward && (aligned || s.cols == 8) ? 1 : 0);
    groups = (n_rows + kWarps - 1) / kWarps;
  } else {
    int most;  // threads per SM
    if (!aligned) {
      s.cols = !forward && n_cols > 16 * 256 && n_cols <= 8 * 640 ? 8
               : n_cols <= 16 * 512                                ? 16
               : n_cols <= 24 * 512                                ? 24
                                                                   : 0;
      most = s.cols != 24 && (forward || s.cols == 8) ? 1024 : 512;
    } else if (forward) {
      s.cols = n_cols < 2048 || xs == 4 ? 16 : n_cols <= 32 * 256 ? 32 : 16;
      if (n_cols > 16 * 768) s.cols = n_cols <= 32 * 512 ? 32 : 0;
      most = s.cols == 32 ? 512 : 768;
    } else {
      const bool two = n_cols <= 32 * 256 &&  // CTAs of 32 columns per thread
                       2 * (size_t)n_cols * (xs + ys) <= kSmemPerSm / 2 - kSmemStatic;
      s.cols = n_cols <= 2048       ? 8
               : n_cols <= 16 * 384 ? 16
               : two                ? 32
               : n_cols <= 16 * 768 ? 16
               : n_cols <= 32 * 512 ? 32
                                    : 0;
      most = s.cols == 32 ? 512 : s.cols == 8 && xs == 4 ? 640 : 768;
    }
    if (!s.cols) return s;
    s.threads = ((n_cols + s.cols - 1) / s.cols + 31) / 32 * 32;
    per_sm = most / s.threads < 1 ? 1 : most / s.threads;
  }
  s.grid = (int)(groups < (int64_t)per_sm * kSms ? groups : (int64_t)per_sm * kSms);
  return s;
}

// Whether dweight and dbias are summed by columns in the launch that makes dx,
// rather than from partial sums of its rows: x and dy are read twice, the
// second time from L2, but there is one launch and no workspace. In us, by
// columns against by rows, fp32 x: 64 x 2048 4.3 / 6.3, 512 x 4096 12.7 /
// 13.7, 1024 x 2048 14.4 / 14.5; beyond these bounds 300 x 8192 16.4 / 13.8,
// 2048 x 1024 18.4 / 15.0.
bool by_columns(int64_t n_rows, int n_cols) {
  return n_rows <= 1024 && n_rows * n_cols <= (9 << 18) && n_cols <= 16 * 512;
}

constexpr int kMaxCols = INT32_MAX - 4096;
constexpr int kRowGrid = kSms * 8;

// Partial sums of dweight and dbias, at most (whichever kernel runs).
int64_t backward_workspace(int64_t n_rows, int n_cols, bool want_params) {
  if (!want_params || n_rows == 0 || by_columns(n_rows, n_cols)) return 0;
  int64_t parts = kLongParts;
  for (const bool aligned : {false, true})
    for (const int xs : {2, 4})
      for (const int ys : {2, 4}) {
        const RowShape s = row_shape(n_rows, n_cols, xs, ys, aligned, false);
        if (s.cols && s.grid > parts) parts = s.grid;
      }
  return parts * 2 * n_cols * 4;
}

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

template <typename Args>
spmv_status launch_rows(void (*fn)(Args), const RowShape& s, size_t smem, const Args& p,
                        cudaStream_t st, int more_ctas = 0) {
  if (!allow_smem(reinterpret_cast<const void*>(fn), smem)) return SPMV_ERR_CUDA;
  return launch(fn, dim3((unsigned)(s.grid + more_ctas)), s.threads, smem, st, p);
}

// Vectors are 16 bytes of x; rows that they do not fit take the same columns
// per thread element by element.
template <typename XT, typename YT, int CPT, bool WARP, bool ALIGNED>
spmv_status forward_launch(const RowShape& s, const ForwardArgs<XT, YT>& p, cudaStream_t st) {
  constexpr int kVec = 16 / (int)sizeof(XT);
  const size_t vectors = (size_t)s.threads * CPT;
  if constexpr (!ALIGNED) {  // weight and bias
    return launch_rows(layernorm_fused<XT, YT, kVec, CPT, 0, WARP>, s, vectors * 8, p, st);
  } else {
    // Two rows on their way where two CTAs share an SM, three where there is
    // one (16384 rows of fp32, 4096 columns: 62 us with two, 65 with three;
    // 8192: 137 with two, 128 with three).
    if constexpr (CPT == 16 && !WARP)
      if (2 * s.threads <= most_threads(16, true))
        return launch_rows(layernorm_fused<XT, YT, kVec, 16, 2, false>, s,
                           2 * vectors * sizeof(XT), p, st);
    constexpr int kStages = WARP ? 4 : 3;
    return launch_rows(layernorm_fused<XT, YT, kVec, CPT, kStages, WARP>, s,
                       kStages * vectors * sizeof(XT), p, st);
  }
}

template <typename XT, typename YT, bool ALIGNED>
spmv_status forward(const ForwardArgs<XT, YT>& p, cudaStream_t st) {
  RowShape s = row_shape(p.n_rows, p.n_cols, sizeof(XT), sizeof(YT), ALIGNED, true);
  if (s.warp)
    return s.cols == 8 ? forward_launch<XT, YT, 8, true, ALIGNED>(s, p, st)
                       : forward_launch<XT, YT, 16, true, ALIGNED>(s, p, st);
  if constexpr (ALIGNED)
    if (s.cols == 32) return forward_launch<XT, YT, 32, false, true>(s, p, st);
  if (s.cols == 16) return forward_launch<XT, YT, 16, false, ALIGNED>(s, p, st);
  if constexpr (!ALIGNED)
    if (s.cols == 24) return forward_launch<XT, YT, 24, false, false>(s, p, st);
  s.threads = kThreads;
  s.grid = (int)(p.n_rows < kRowGrid ? p.n_rows : kRowGrid);
  return launch_rows(layernorm_rows<XT, YT>, s, 0, p, st);
}

template <typename XT, typename YT, int CPT, bool WARP, bool ALIGNED>
spmv_status backward_launch(const RowShape& s, const BackwardArgs<XT, YT>& p, cudaStream_t st) {
  constexpr int kVec = 16 / (int)sizeof(XT);
  const int columns = p.dweight || p.dbias ? (p.n_cols + 31) / 32 : 0;  // CTAs for them
  if constexpr (!ALIGNED) {
    return launch_rows(layernorm_backward_fused<XT, YT, kVec, CPT, 0, 1, WARP>, s,
                       (size_t)s.threads * CPT * 4, p, st, columns);
  } else {
    // Two rows at a time halve the barriers (a warp's rows need none; 8192 x
    // 12288 bf16: 120 us, single rows 131); where two sets of them do not fit,
    // single rows. (A warp group's ring is larger than the two sums per column
    // that the warps leave in its place at the end.)
    const size_t row = (size_t)s.threads * CPT * (sizeof(XT) + sizeof(YT));
    const size_t room =
        kSmemPerSm / (size_t)((s.grid + columns + kSms - 1) / kSms) - kSmemStatic;
    if constexpr (CPT < 32) {
      if constexpr (!WARP)
        if (4 * row <= room)
          return launch_rows(layernorm_backward_fused<XT, YT, kVec, CPT, 2, 2, false>, s, 4 * row,
                             p, st, columns);
      if (3 * row <= room)
        return launch_rows(layernorm_backward_fused<XT, YT, kVec, CPT, 3, 1, WARP>, s, 3 * row, p,
                           st, columns);
    }
    return launch_rows(layernorm_backward_fused<XT, YT, kVec, CPT, 2, 1, WARP>, s, 2 * row, p, st,
                       columns);
  }
}

template <typename XT, typename YT, bool ALIGNED>
spmv_status backward(BackwardArgs<XT, YT> p, void* dweight, void* dbias, cudaStream_t st) {
  RowShape s = row_shape(p.n_rows, p.n_cols, sizeof(XT), sizeof(YT), ALIGNED, false);
  const bool columns = (dweight || dbias) && by_columns(p.n_rows, p.n_cols);
  // two sets of 32 columns' rows in fp32 do not fit shared memory
  if (s.cols == 32 && ALIGNED &&
      2 * (size_t)s.threads * 32 * (sizeof(XT) + sizeof(YT)) > kSmemPerSm - kSmemStatic)
    s.cols = 0;
  if (columns) {
    p.part = nullptr;
    // CTAs of 16 warps at least, for the columns' rows
    if (s.warp || (s.cols == 16 && p.n_cols <= 8 * 640)) {
      s.warp = false;
      s.cols = 8;
      s.threads = ((p.n_cols + 7) / 8 + 31) / 32 * 32;
    } else if (s.cols == 32) {
      s.cols = 16;
    }
    if (s.threads < 512) s.threads = 512;
    const int64_t most = s.cols == 8 ? 2 * kSms : kSms;
    s.grid = (int)(p.n_rows < most ? p.n_rows : most);
    if (p.dx == static_cast<const void*>(p.dy)) {  // the columns first: dx takes dy's place
      BackwardArgs<XT, YT> q = p;
      q.dx = nullptr;
      const spmv_status status = backward<XT, YT, ALIGNED>(q, dweight, dbias, st);
      if (status != SPMV_OK) return status;
    } else {
      p.dweight = dweight, p.dbias = dbias;
    }
    if (!p.dx) s.grid = 0;
  }
  p.row_ctas = s.grid;
  int parts = s.grid;
  spmv_status status = SPMV_OK;
  if (s.warp) {
    status = s.cols == 8 ? backward_launch<XT, YT, 8, true, ALIGNED>(s, p, st)
                         : backward_launch<XT, YT, 16, true, ALIGNED>(s, p, st);
  } else if (s.cols == 8) {
    status = backward_launch<XT, YT, 8, false, ALIGNED>(s, p, st);
  } else if (s.cols == 16) {
    status = backward_launch<XT, YT, 16, false, ALIGNED>(s, p, st);
  } else if (s.cols) {
    status = backward_launch<XT, YT, ALIGNED ? 32 : 24, false, ALIGNED>(s, p, st);
  } else {
    const int grid = (int)(p.n_rows < kRowGrid ? p.n_rows : kRowGrid);
    parts = kLongParts;
    if (p.part)
      status = launch(layernorm_params_part<XT, YT>,
                      dim3((unsigned)((p.n_cols + kThreads - 1) / kThreads), kLongParts), kThreads,
                      0, st, p);
    if (p.dx && status == SPMV_OK)
      status = launch(layernorm_dx_rows<XT, YT>, dim3((unsigned)grid), kThreads, 0, st, p);
  }
  if (status != SPMV_OK || !p.part) return status;
  int n_cols = p.n_cols, pt = p.pt;
  const float* part = p.part;
  void* args[] = {&n_cols, &parts, &part, &dweight, &dbias, &pt};
  return status_of_launch(launch_pdl(reinterpret_cast<const void*>(&layernorm_params_sum),
                                     (int)((2ll * n_cols + 31) / 32), kSumWarps * 32, 0, st,
                                     args));
}

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
  return by_types(x_dtype, y_dtype, [&](auto* xt, auto* yt) {
    using XT = std::remove_pointer_t<decltype(xt)>;
    using YT = std::remove_pointer_t<decltype(yt)>;
    constexpr int kVec = 16 / (int)sizeof(XT);
    const ForwardArgs<XT, YT> p{n_rows, n_cols, static_cast<const XT*>(x), x_stride, weight, bias,
                                param_dtype, eps, static_cast<YT*>(y), y_stride, mean_out,
                                rstd_out};
    // whole vectors need every row of x and y, weight and bias on vector
    // boundaries and a whole number of vectors per row
    if (n_cols % kVec == 0 && rows_aligned(x, n_rows, x_stride, xs, kVec) &&
        rows_aligned(y, n_rows, y_stride, ysz, kVec) && aligned_to(weight, 16) &&
        aligned_to(bias, 16))
      return forward<XT, YT, true>(p, st);
    return forward<XT, YT, false>(p, st);
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
    spmv_status status = SPMV_OK;
    for (void* sum : {dweight, dbias})
      if (sum && status == SPMV_OK)
        status = status_of(cudaMemsetAsync(sum, 0, (size_t)(n_cols * ps), st));
    return status;
  }
  return by_types(x_dtype, dy_dtype, [&](auto* xt, auto* yt) {
    using XT = std::remove_pointer_t<decltype(xt)>;
    using YT = std::remove_pointer_t<decltype(yt)>;
    constexpr int kVec = 16 / (int)sizeof(XT);
    BackwardArgs<XT, YT> p{n_rows, n_cols, static_cast<const YT*>(dy), dy_stride,
                           static_cast<const XT*>(x), x_stride, weight, param_dtype, mean, rstd,
                           static_cast<XT*>(dx), dx_stride,
                           params ? static_cast<float*>(workspace) : nullptr, 0, nullptr,
                           nullptr};
    if (n_cols % kVec == 0 && rows_aligned(x, n_rows, x_stride, xs, kVec) &&
        rows_aligned(dy, n_rows, dy_stride, dys, kVec) &&
        (!dx || rows_aligned(dx, n_rows, dx_stride, xs, kVec)) && aligned_to(weight, 16))
      return backward<XT, YT, true>(p, dweight, dbias, st);
    return backward<XT, YT, false>(p, dweight, dbias, st);
  });
}
