// Rotary positions of queries and keys (fs_rope): pair (x, y) of a head turned by the
// angle a = position * frequency, to factor * (x cos a - y sin a, y cos a + x sin a).
//
// Angles. A frequency is held as a 64-bit fraction of a turn a position, F = f / (2 pi) *
// 2^64; position * F modulo 2^64 is the angle's fraction of a turn, exact but for F's
// rounding (position * 2^-65 turns), whatever the position: whole turns drop out of the
// integer product. (f64 would cost more than the rows' bytes do: its rate here is 1/60 of
// f32's.) The signed top 24 bits give sine and cosine by sincospi, the next 24 turn them
// by a first-order step, as their angle is below 2^-21 (2 pi 2^-24); the last 16, below 2^-48
// turns, are left out.
//
// One pass over the bytes, which bound it: a thread has one vector of pairs of a row, computes
// their sines and cosines once and takes several heads by them. 65536 rows of 40 heads of 128
// in bf16: 207 us, 6.5 TB/s, 0.96 of the measured copy; 4099 rows of 18 heads of 256 in f32, a
// quarter turned: 25 us, 0.88; one row: 2 us, the launch.
#include "fs_internal.h"

namespace fsk {
namespace {

template <int kBytes>
struct VecOf;
template <>
struct VecOf<16> { using T = uint4; };
template <>
struct VecOf<4> { using T = uint32_t; };
template <>
struct VecOf<2> { using T = uint16_t; };

// kN consecutive values of T in vectors of kBytes; kStream: the caches keep them no longer
// than others.
template <typename T, int kN, int kBytes, bool kStream>
struct Vals {
  using V = typename VecOf<kBytes>::T;
  static constexpr int kV = kN * (int)sizeof(T) / kBytes;
  V v[kV];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      const V* q = reinterpret_cast<const V*>(p) + i;
      v[i] = kStream ? __ldcs(q) : *q;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kV; ++i) {
      V* q = reinterpret_cast<V*>(p) + i;
      if (kStream) __stcs(q, v[i]);
      else *q = v[i];
    }
  }
  __device__ __forceinline__ float get(int i) const {
    const T x = reinterpret_cast<const T*>(v)[i];
    if constexpr (sizeof(T) == 4) return x;
    else return __bfloat162float(x);
  }
  __device__ __forceinline__ void set(int i, float x) {
    T* p = reinterpret_cast<T*>(v);
    if constexpr (sizeof(T) == 4) p[i] = x;
    else p[i] = __float2bfloat16_rn(x);
  }
};

// (cos, sin) of pos * F turns, times m.
__device__ __forceinline__ float2 turn(uint32_t pos, uint64_t F, float m, bool inverse) {
  const uint64_t r = (uint64_t)pos * F;
  const int top = (int)(r >> 32) >> 8;               // of 2^-24 turns, signed
  const float rest = (float)((uint32_t)(r >> 16) & 0xffffffu);  // of 2^-48 turns
  float s, c;
  sincospif((float)top * 0x1p-23f, &s, &c);
  const float d = rest * (6.2831855f * 0x1p-48f);
  const float s1 = fmaf(c, d, s), c1 = fmaf(-s, d, c);
  return make_float2(c1 * m, (inverse ? -s1 : s1) * m);
}

// kNear: pairs of neighbours, else of halves. A unit is kP pairs of a head, or 2 kP
// values behind the turned ones, which are copied.
template <typename T, int kBytes, bool kNear, bool kStream>
__global__ void __launch_bounds__(256) k_rope(const RopeArgs a) {
  constexpr int kP = kNear ? (kBytes / (2 * (int)sizeof(T)) > 0 ? kBytes / (2 * (int)sizeof(T)) : 1)
                           : kBytes / (int)sizeof(T);
  pdl_wait();
  pdl_trigger();
  const int half = a.rot / 2, turned = half / kP;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t item = t / a.units;  // (row, group of heads)
  const int unit = (int)(t - item * a.units);
  const int row = (int)(item / a.groups), group = (int)(item - (int64_t)row * a.groups);
  if (row >= a.n) return;
  const int pos = a.positions[row];
  if (pos < 0) return;
  const int H = a.H + a.Hkv;
  const int h0 = group * a.per, h1 = min(H, h0 + a.per);
  auto in = [&](int h) {
    return h < a.H ? static_cast<const T*>(a.q) + row * a.q_stride + (int64_t)h * a.hd
                   : static_cast<const T*>(a.k) + row * a.k_stride + (int64_t)(h - a.H) * a.hd;
  };
  auto out = [&](int h) {
    return h < a.H ? static_cast<T*>(a.q_out) + row * a.qo_stride + (int64_t)h * a.hd
                   : static_cast<T*>(a.k_out) + row * a.ko_stride + (int64_t)(h - a.H) * a.hd;
  };
  // kH heads at a time: their loads, eight, are asked for before the first store (4099 rows
  // of neighbours: 25 us, with four loads 27; 65536 rows of halves: 207 us, with sixteen 202)
  constexpr int kH = kNear ? 8 : 4;
  if (unit >= turned) {  // behind the turned values (out of place)
    constexpr int kE = kBytes / (int)sizeof(T);
    const int at = a.rot + (unit - turned) * kE;
#pragma unroll 1
    for (int h = h0; h < h1; h += 8) {
      Vals<T, kE, kBytes, kStream> x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (h + u < h1) x[u].load(in(h + u) + at);
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (h + u < h1) x[u].store(out(h + u) + at);
    }
    return;
  }
  float2 cs[kP];
#pragma unroll
  for (int i = 0; i < kP; ++i) cs[i] = turn((uint32_t)pos, a.F[unit * kP + i], a.factor, a.inverse);
#pragma unroll 1
  for (int h = h0; h < h1; h += kH) {
    if constexpr (kNear) {
      Vals<T, 2 * kP, kBytes, kStream> x[kH];
#pragma unroll
      for (int u = 0; u < kH; ++u)
        if (h + u < h1) x[u].load(in(h + u) + unit * 2 * kP);
#pragma unroll
      for (int u = 0; u < kH; ++u) {
        if (h + u >= h1) break;
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          const float v = x[u].get(2 * i), w = x[u].get(2 * i + 1);
          x[u].set(2 * i, fmaf(v, cs[i].x, -w * cs[i].y));
          x[u].set(2 * i + 1, fmaf(w, cs[i].x, v * cs[i].y));
        }
        x[u].store(out(h + u) + unit * 2 * kP);
      }
    } else {
      Vals<T, kP, kBytes, kStream> x[kH], y[kH];
#pragma unroll
      for (int u = 0; u < kH; ++u)
        if (h + u < h1) {
          x[u].load(in(h + u) + unit * kP);
          y[u].load(in(h + u) + half + unit * kP);
        }
#pragma unroll
      for (int u = 0; u < kH; ++u) {
        if (h + u >= h1) break;
#pragma unroll
        for (int i = 0; i < kP; ++i) {
          const float v = x[u].get(i), w = y[u].get(i);
          x[u].set(i, fmaf(v, cs[i].x, -w * cs[i].y));
          y[u].set(i, fmaf(w, cs[i].x, v * cs[i].y));
        }
        x[u].store(out(h + u) + unit * kP);
        y[u].store(out(h + u) + half + unit * kP);
      }
    }
  }
}

template <typename T, int kBytes>
Launched launch_t(RopeArgs a, bool near, int sms, cudaStream_t s) {
  constexpr int kE = kBytes / (int)sizeof(T);
  const int p = near ? std::max(1, kE / 2) : kE;
  const bool copies = a.q_out != a.q || (a.Hkv > 0 && a.k_out != a.k);
  a.units = a.rot / 2 / p + (copies ? (a.hd - a.rot) / kE : 0);
  // heads a thread: all, or as few as fill the SMs' threads (latency)
  const int heads = a.H + a.Hkv;
  const int64_t fill = (int64_t)sms * 2048 / std::max<int64_t>(1, (int64_t)a.n * a.units);
  a.groups = (int)std::min<int64_t>(heads, std::max<int64_t>(1, fill));
  a.per = (heads + a.groups - 1) / a.groups;
  a.groups = (heads + a.per - 1) / a.per;
  const int64_t threads = (int64_t)a.n * a.groups * a.units;
  // what is more than the L2 may keep passes through it first to go (65536 rows, 537 MB and as
  // much out: 207 us, without 230; 4099 rows, 75 MB: 25 and 27)
  constexpr bool kWide = kBytes == 16;
  const bool stream = kWide && (int64_t)a.n * heads * a.hd * (int64_t)sizeof(T) > (64 << 20);
  auto kernel = stream ? (near ? k_rope<T, kBytes, true, kWide> : k_rope<T, kBytes, false, kWide>)
                       : (near ? k_rope<T, kBytes, true, false> : k_rope<T, kBytes, false, false>);
  Launched l;
  l.add(launch_k(kernel, dim3((unsigned)((threads + 255) / 256)), 256, 0, s, a));
  return l;
}

// The widest vectors that every row, head, half and the copied rest start and end on.
template <typename T>
Launched launch_x(const RopeArgs& a, bool near, int sms, cudaStream_t s) {
  const int64_t e = sizeof(T);
  int64_t all = (int64_t)reinterpret_cast<uintptr_t>(a.q) | (int64_t)reinterpret_cast<uintptr_t>(a.q_out) |
                a.hd * e | a.rot * e | (near ? 0 : a.rot / 2 * e);
  if (a.n > 1) all |= a.q_stride * e | a.qo_stride * e;
  if (a.Hkv) {
    all |= (int64_t)reinterpret_cast<uintptr_t>(a.k) | (int64_t)reinterpret_cast<uintptr_t>(a.k_out);
    if (a.n > 1) all |= a.k_stride * e | a.ko_stride * e;
  }
  if (all % 16 == 0) return launch_t<T, 16>(a, near, sms, s);
  if (sizeof(T) == 4 || all % 4 == 0) return launch_t<T, 4>(a, near, sms, s);
  if constexpr (sizeof(T) == 2) return launch_t<T, 2>(a, near, sms, s);
  return {};
}

}  // namespace

Launched launch_rope(const RopeArgs& a, int x_type, bool near, int sms, cudaStream_t s) {
  return x_type == X_F32 ? launch_x<float>(a, near, sms, s) : launch_x<__nv_bfloat16>(a, near, sms, s);
}

}  // namespace fsk
