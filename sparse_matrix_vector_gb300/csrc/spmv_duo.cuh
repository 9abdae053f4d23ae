// Numbers as unevaluated sums of two fp32 (some 2^-47 of relative error each
// operation), for what lies next to a border: sums of exponentials whose
// comparison with a given random number has to come out as in 64 bits. The
// device's fp64 rate is a sixtieth of its fp32 rate; these cost some twenty
// fp32 operations. The sums and products are the error-free transformations
// of Dekker (1971) and Knuth, with fused multiply-adds for the products.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace spmv {
namespace {

struct Duo {
  float h, l;
};

__device__ __forceinline__ Duo fast_two_sum(float a, float b) {  // |a| >= |b|, or a = 0
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Duo two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Duo duo_add(const Duo& a, const Duo& b) {
  const Duo s = two_sum(a.h, b.h);
  return fast_two_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Duo duo_mul(const Duo& a, const Duo& b) {
  const float p = __fmul_rn(a.h, b.h);
  const float e = __fmaf_rn(a.h, b.h, -p);
  return fast_two_sum(p, __fadd_rn(e, __fmaf_rn(a.h, b.l, __fmul_rn(a.l, b.h))));
}
__device__ __forceinline__ Duo duo_of(double v) {
  const float h = (float)v;
  return {h, (float)(v - (double)h)};
}
__device__ __forceinline__ double to_f64(const Duo& a) { return (double)a.h + (double)a.l; }

// 2^(j / 64), to 2^-48.
__device__ const float2 kRoots[64] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.02c9a40000000p+0f, -0x1.887fa00000000p-28f},
    {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f}, {0x1.0874520000000p+0f, -0x1.e2990e0000000p-26f},
    {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f}, {0x1.0e3ec40000000p+0f, -0x1.a585cc0000000p-25f},
    {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f}, {0x1.1429aa0000000p+0f, 0x1.d525bc0000000p-25f},
    {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.1a35be0000000p+0f, 0x1.6df96e0000000p-25f},
    {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f}, {0x1.2063b80000000p+0f, 0x1.0c519a0000000p-25f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.26b4560000000p+0f, 0x1.789f380000000p-26f},
    {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f}, {0x1.2d285a0000000p+0f, 0x1.b900c20000000p-26f},
    {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}, {0x1.33c08c0000000p+0f, -0x1.b37d200000000p-25f},
    {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f}, {0x1.3a7db40000000p+0f, -0x1.634c020000000p-25f},
    {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}, {0x1.4160a20000000p+0f, 0x1.f72e2a0000000p-28f},
    {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f}, {0x1.486a2c0000000p+0f, -0x1.47d8660000000p-25f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.4f9b280000000p+0f, -0x1.2c5a6c0000000p-25f},
    {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f}, {0x1.56f4740000000p+0f, -0x1.295b040000000p-25f},
    {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f}, {0x1.5e76f20000000p+0f, -0x1.4a5bd60000000p-25f},
    {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f}, {0x1.6623880000000p+0f, 0x1.2a91120000000p-27f},
    {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.6dfb240000000p+0f, -0x1.cd72e80000000p-27f},
    {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f}, {0x1.75feb60000000p+0f, -0x1.37b3060000000p-25f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.7e2f340000000p+0f, -0x1.2616340000000p-25f},
    {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f}, {0x1.868d9a0000000p+0f, -0x1.2edb440000000p-26f},
    {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f}, {0x1.8f1aea0000000p+0f, -0x1.baa2320000000p-26f},
    {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f}, {0x1.97d82a0000000p+0f, -0x1.0d8d840000000p-31f},
    {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}, {0x1.a0c6680000000p+0f, -0x1.2886a60000000p-26f},
    {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f}, {0x1.a9e6b60000000p+0f, -0x1.50c0480000000p-25f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b33a2c0000000p+0f, -0x1.ec3a820000000p-26f},
    {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f}, {0x1.bcc1ea0000000p+0f, -0x1.f687c60000000p-25f},
    {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f}, {0x1.c67f120000000p+0f, 0x1.cafa2a0000000p-25f},
    {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f}, {0x1.d072d40000000p+0f, 0x1.40f1300000000p-25f},
    {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.da9e600000000p+0f, 0x1.ed99420000000p-27f},
    {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f}, {0x1.e502ee0000000p+0f, 0x1.e2cffe0000000p-26f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.efa1be0000000p+0f, 0x1.cc2b440000000p-25f},
    {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f}, {0x1.fa7c180000000p+0f, 0x1.9e90d80000000p-28f},};

// 2^a for a <= 0, to some 2^-40; 0 below 2^-126. With k = round(64 a),
// 2^a = 2^(k / 64) e^y, |y| <= log(2) / 128: a table (Tang 1989) and five
// terms of the exponential's series. `roots`: kRoots in shared memory.
__device__ __forceinline__ Duo duo_exp2(const Duo& a, const float2* roots) {
  if (!(a.h >= -126.f)) return {0.f, 0.f};
  const float k = rintf(a.h * 64.f);
  const Duo g = two_sum(__fmaf_rn(k, -1.f / 64.f, a.h), a.l);  // (the difference is exact)
  const float ln2_h = 0x1.62e43p-1f, ln2_l = -0x1.05c61p-29f;
  const float yh = __fmul_rn(g.h, ln2_h);
  const float yl = __fadd_rn(__fmaf_rn(g.h, ln2_h, -yh), __fmaf_rn(g.h, ln2_l, __fmul_rn(g.l, ln2_h)));
  // e^y - 1 - yh
  float q = __fmaf_rn(yh, 1.f / 120.f, 1.f / 24.f);
  q = __fmaf_rn(q, yh, 1.f / 6.f);
  q = __fmaf_rn(q, yh, 0.5f);
  q = __fmul_rn(q, __fmul_rn(yh, yh));
  q = __fadd_rn(q, __fmaf_rn(yh, yl, yl));
  const Duo e = fast_two_sum(1.f, yh);
  const int ki = (int)k;
  const float2 r = roots[ki & 63];
  const Duo p = duo_mul({e.h, __fadd_rn(e.l, q)}, {r.x, r.y});
  const float up = __int_as_float(((ki >> 6) + 127) << 23);  // 2^floor(k / 64), at least 2^-126
  return {__fmul_rn(p.h, up), __fmul_rn(p.l, up)};
}

}  // namespace
}  // namespace spmv
