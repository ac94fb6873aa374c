// Numbers of about 46 bits as unevaluated sums of two f32 (Dekker 1971; Knuth's
// two-sum), for decisions that lie next to a border: the f64 units of this GPU run
// at 1/60 of its f32 rate.
#pragma once

namespace fsk {
namespace two {

// An unevaluated sum h + l of two f32 numbers, |l| at most half a last place of h.
struct Two {
  float h, l;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ Two fast_two_sum(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ Two add(Two a, Two b) {
  const Two s = two_sum(a.h, b.h);
  return fast_two_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Two two_prod(float a, float b) {  // exact
  const float p = __fmul_rn(a, b);
  return {p, fmaf(a, b, -p)};
}
__device__ __forceinline__ Two mul(Two a, Two b) {
  const float p = __fmul_rn(a.h, b.h);
  return fast_two_sum(p, fmaf(a.h, b.h, -p) + fmaf(a.h, b.l, __fmul_rn(a.l, b.h)));
}
__device__ __forceinline__ bool less(Two a, Two b) {
  return a.h < b.h || (a.h == b.h && a.l < b.l);
}

}  // namespace two
}  // namespace fsk
