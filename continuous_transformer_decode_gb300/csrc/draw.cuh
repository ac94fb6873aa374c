// Weights exp((z - max) / T) of logits, and the pieces of a draw from them: what
// verification of drafts (k_verify.cu) and sampling (k_sample_filtered.cu) share.
#pragma once

#include <math_constants.h>

#include "two_f32.cuh"

namespace fsk {
namespace draw {

using namespace two;

constexpr unsigned kAll = 0xffffffffu;

// 2^(k/32) as pairs of f32 numbers.
static __constant__ float2 kExp2[32] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f},
    {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f}, {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f},
    {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f},
    {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}, {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f},
    {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}, {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f},
    {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f}, {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f},
    {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f},
    {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f}, {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f},
    {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}, {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f},
    {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f}, {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f},
    {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f}};

__device__ __forceinline__ Two shfl_xor(Two v, int o) {
  return {__shfl_xor_sync(0xffffffffu, v.h, o), __shfl_xor_sync(0xffffffffu, v.l, o)};
}
// log2(e) / T
__device__ __forceinline__ Two log2e_over(float T) {
  const float lh = 1.4426950216293335f, ll = 1.9259629911266175e-08f;
  const float q = lh / T;
  return {q, (fmaf(-q, T, lh) + ll) / T};
}

// 2^60 exp((z - m) / T) as 2^(60 + y), y = (z - m) * c with c = log2(e) / T, to a
// relative 2^-36: y = n + k/32 + f with |f| <= 1/64, 2^f = 1 + its Taylor series (the
// method of Tang, ACM TOMS 1989). Below y = -125.5 it is zero. The factor, which every
// weight and sum in pairs has, keeps the second halves of the smallest (2^-150 of the
// largest) in f32's range, and the largest sum, 2^30 of them, as well.
constexpr float kUp = 0x1p60f;
__device__ __forceinline__ Two weight2(float z, float m, Two c, const float2* tab) {
  const Two d = two_sum(z, -m);
  const float p = __fmul_rn(d.h, c.h);
  const float pe = fmaf(d.h, c.h, -p) + fmaf(d.h, c.l, __fmul_rn(d.l, c.h));
  const float kf = rintf(__fmul_rn(p, 32.0f));
  const int k = (int)kf;
  const float fh = fmaf(kf, -0.03125f, p), fl = pe;  // fh is exact
  const float f = __fadd_rn(fh, fl);
  const float l1h = 0.6931471824645996f, l1l = -1.9046542e-09f;  // ln 2
  const float a = __fmul_rn(fh, l1h);
  const float ae = fmaf(fh, l1h, -a) + fmaf(fh, l1l, __fmul_rn(fl, l1h));
  float q = fmaf(f, 0.0013333558f, 0.009618129f);  // ln2^5 / 5!, ln2^4 / 4!
  q = fmaf(f, q, 0.05550411f);
  q = fmaf(f, q, 0.2402265f);
  const Two u = fast_two_sum(a, fmaf(__fmul_rn(f, f), q, ae));  // 2^f - 1
  const float2 t = tab[k & 31];
  const float w = __fmul_rn(t.x, u.h);
  const float we = fmaf(t.x, u.h, -w) + fmaf(t.x, u.l, fmaf(t.y, u.h, t.y));
  const Two e = fast_two_sum(t.x, w);
  const Two r = fast_two_sum(e.h, __fadd_rn(e.l, we));
  const float s = __int_as_float(((k >> 5) + 127 + 60) << 23);  // 2^60 2^n, -126 <= n <= 0
  // no branches: several of these run interleaved
  const bool one = z == m, in = p > -125.5f;  // not in: also -inf and NaN
  return {one ? kUp : in ? __fmul_rn(r.h, s) : 0.0f, !one && in ? __fmul_rn(r.l, s) : 0.0f};
}

// f32 weight under m; c = log2(e) / T. Good to a relative (4 + 1.4 |y|) 2^-24 with y
// its logarithm to the base 2: ex2.approx is good to 2^-22, and z - m and then y are
// rounded, 2^-24 |y| each, times ln 2. Zero below y = -126.
__device__ __forceinline__ float weight1(float z, float m, Two c) {
  if (m == CUDART_INF_F) return z == m ? 1.0f : 0.0f;
  const float d = z - m;
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(fmaxf(fmaf(d, c.h, d * c.l), -200.0f)));
  return y;  // 0 for NaN and -inf
}
// factor that takes sums under m to sums under M
__device__ __forceinline__ float rescale(float m, float M, Two c) {
  return m == -CUDART_INF_F ? 0.0f : m == M ? 1.0f : weight1(m, M, c);
}

__device__ __forceinline__ float4 load4(const float* z, int i, int hi, bool vec) {
  if (vec && i + 4 <= hi) return *reinterpret_cast<const float4*>(z + i);
  float4 v = make_float4(-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F);
  if (i < hi) v.x = z[i];
  if (i + 1 < hi) v.y = z[i + 1];
  if (i + 2 < hi) v.z = z[i + 2];
  if (i + 3 < hi) v.w = z[i + 3];
  return v;
}

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ Two shfl_up(Two v, int o) {
  return {__shfl_up_sync(kAll, v.h, o), __shfl_up_sync(kAll, v.l, o)};
}
__device__ __forceinline__ Two shfl(Two v, int i) {
  return {__shfl_sync(kAll, v.h, i), __shfl_sync(kAll, v.l, i)};
}
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float shfl_up(float v, int o) { return __shfl_up_sync(kAll, v, o); }
__device__ __forceinline__ float shfl(float v, int i) { return __shfl_sync(kAll, v, i); }
__device__ __forceinline__ bool less(float a, float b) { return a < b; }
__device__ __forceinline__ bool positive(float a) { return a > 0.0f; }
__device__ __forceinline__ bool positive(Two a) { return a.h > 0.0f; }

// Inclusive sums over the lanes.
template <typename T>
__device__ __forceinline__ T scan(T v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T up = shfl_up(v, o);
    if (lane >= o) v = add(up, v);
  }
  return v;
}
// Of parts with weights, two a lane, the first whose running sum reaches the target, or
// the last with a weight, or -1; `before` becomes the sum of those ahead of it.
template <typename T>
__device__ __forceinline__ int pick(T w0, T w1, T target, T& before, int lane) {
  const T upto = scan(add(w0, w1), lane);
  const bool some = positive(w0) || positive(w1);
  const unsigned has = __ballot_sync(kAll, some);
  const unsigned hit = __ballot_sync(kAll, some && !less(upto, target));
  if (!has) return -1;
  const int at = hit ? __ffs(hit) - 1 : 31 - __clz(has);
  if (at > 0) before = shfl(upto, at - 1);
  w0 = shfl(w0, at);
  w1 = shfl(w1, at);
  const T half = add(before, w0);
  if (positive(w0) && (!positive(w1) || (hit && !less(half, target)))) return 2 * at;
  before = half;
  return 2 * at + 1;
}

}  // namespace draw
}  // namespace fsk
