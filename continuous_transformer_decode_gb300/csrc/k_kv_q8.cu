// Quantised writes into the 8-bit paged KV cache, and reads back out of it.
//
// A row x of hd values (one token, one KV head; keys after their rotation)
// is stored as scale = amax / 127 and codes round(x * 127 / amax), ties to
// even, amax the largest magnitude; a value stands for code * scale.
//
// The bytes are each value in and its code out, or the reverse. hd / 8 lanes share a
// row, each with four values of its lower and four of its upper half (what a
// rotation pairs), so that the loads and stores of a warp are whole sectors of
// consecutive rows, and every lane has its key and its value row in flight
// together. 65536 rows of 8 heads of 128 in bf16 are read back in 73 us, 5.6 TB/s, and
// written in 104 us, 3.9 TB/s: 381 instructions for a warp's two rows of keys and two of
// values bound that (0.79 of the issue slots). Rounding to a code is one fused multiply-add: x * r + 1.5 * 2^23 + 128
// has the byte code + 128 in its last bits.

#include <float.h>

#include <type_traits>

#include "kv_q8.cuh"
#include "two_f32.cuh"

namespace fsk {
FS_TRACE_TU(kv_q8)
namespace {

using namespace two;

constexpr int kT = 128;
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Four consecutive elements; kVec: their address is aligned to all four.
template <bool kVec>
__device__ __forceinline__ void load4(const float* p, float x[4]) {
  if constexpr (kVec) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  } else {
    x[0] = p[0], x[1] = p[1], x[2] = p[2], x[3] = p[3];
  }
}
template <bool kVec>
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float x[4]) {
  if constexpr (kVec) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
    x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = __bfloat162float(p[j]);
  }
}
template <bool kVec>
__device__ __forceinline__ void store4(float* p, const float x[4]) {
  if constexpr (kVec) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = x[j];
  }
}
// Two values as bf16, those past its range as its largest: the largest f32, which
// stands for a stored infinity, is past it.
__device__ __forceinline__ uint32_t finite_bf16x2(float lo, float hi) {
  uint32_t y;
  asm("cvt.rn.satfinite.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
  return y;
}
template <bool kVec>
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float x[4]) {
  const uint32_t a = finite_bf16x2(x[0], x[1]), b = finite_bf16x2(x[2], x[3]);
  if constexpr (kVec) {
    *reinterpret_cast<uint2*>(p) = make_uint2(a, b);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      p[j] = __ushort_as_bfloat16((unsigned short)((j < 2 ? a : b) >> (16 * (j & 1))));
  }
}

// What a cache row can hold: NaN becomes 0, infinities the largest finite f32.
__device__ __forceinline__ float storable(float x) {
  return x != x ? 0.0f : fminf(fmaxf(x, -FLT_MAX), FLT_MAX);
}
// The largest scale: the f32 below FLT_MAX / 127 rounded, which is above the quotient, so
// that 127 of it would be infinite. Within 2^-23 of the quotient.
constexpr float kMaxScale = 0x1.020406p+121f;
// Largest magnitude of three; NaN if one is.
__device__ __forceinline__ float max_abs(float a, float b, float c) {
  float y;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
__device__ __forceinline__ float max_abs(const float (&x)[8]) {
  return max_abs(max_abs(x[0], x[1], x[2]), max_abs(x[3], x[4], x[5]), max_abs(x[6], x[7], 0.0f));
}

// A quotient in f32 is off by at most kNear of a step: the factor 127 / amax and
// the product round by 2^-24 of at most 127 each, 1.6e-5 together; of a rotated
// key x is off by (1 + sqrt 2) 2^-24 amax, two rounded products and their sum,
// 1.9e-5 of a step, and amax likewise.
template <bool kRot>
constexpr float kNear = kRot ? 6e-5f : 2e-5f;
constexpr float kMagic = 12582912.0f + 128.0f;

// The rows that quantise_row() leaves (of 128 values, one in 200 of f32 and one in 65
// of rotated keys): a quotient may lie on either side of the border of two codes, the
// row is very large or small, or not finite. One warp takes the row and decides by
// comparing 127 x with the border times amax as two-f32 numbers: exactly for
// values that were not rotated, to 2^-44 for others. It is kept out of line and
// loads the row again, so that the other rows do not hold its registers (inlined
// in f64, 65536 rows of 8 heads of 128 took 473 us; inlined so, 179 us).
template <typename T, int HD, bool kRot>
__device__ __noinline__ void quantise_border_row(const T* x, const float* rc, const float* rs,
                                                 uint8_t* codes, float* scale, int lane) {
  constexpr int kHalf = HD / 2, kP = HD / 64;  // pairs (i, i + hd / 2) of a lane
  float a[kP], b[kP], co[kP], si[kP];
#pragma unroll
  for (int p = 0; p < kP; ++p) {
    const int i = lane + 32 * p;
    a[p] = ld1(x + i);
    b[p] = ld1(x + i + kHalf);
    co[p] = kRot ? rc[i] : 1.0f;
    si[p] = kRot ? rs[i] : 0.0f;
  }
  // the two elements of pair p, rounded to f32; and times a power of two as two numbers
  auto rounded = [&](int p, float& y0, float& y1) {
    y0 = a[p], y1 = b[p];
    if constexpr (kRot) rope_pair(a[p], b[p], co[p], si[p], y0, y1);
    y0 = storable(y0), y1 = storable(y1);
  };
  auto exact = [&](int p, int half, float y, float up) -> Two {
    if (!kRot || !(fabsf(y) < FLT_MAX)) return {y * up, 0.0f};
    const float a0 = a[p] * up, b0 = b[p] * up;
    const Two e = half == 0 ? add(two_prod(a0, co[p]), two_prod(b0, -si[p]))
                            : add(two_prod(b0, co[p]), two_prod(a0, si[p]));
    return e.h == e.h ? e : Two{y * up, 0.0f};  // NaN: storable has made it 0
  };
  float amax = 0.0f;
#pragma unroll
  for (int p = 0; p < kP; ++p) {
    float y0, y1;
    rounded(p, y0, y1);
    amax = fmaxf(amax, fmaxf(fabsf(y0), fabsf(y1)));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
  // into the range where quotients and products neither overflow nor vanish
  const float up = amax < 1e-30f ? 0x1p96f : amax > 1e30f ? 0x1p-96f : 1.0f;
  const float top = amax * up, r = top > 0.0f ? 127.0f / top : 0.0f;
  Two y = {0.0f, 0.0f};  // the largest magnitude: of the elements that have it in f32
#pragma unroll
  for (int q = 0; q < 2 * kP; ++q) {
    float v[2];
    rounded(q >> 1, v[0], v[1]);
    const float w = q & 1 ? v[1] : v[0];
    if (fabsf(w) * up >= top * (1.0f - 0x1p-20f)) {
      Two e = exact(q >> 1, q & 1, w, up);
      if (e.h < 0.0f) e = {-e.h, -e.l};
      if (less(y, e)) y = e;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Two e = {__shfl_xor_sync(kAll, y.h, o), __shfl_xor_sync(kAll, y.l, o)};
    if (less(y, e)) y = e;
  }
#pragma unroll
  for (int q = 0; q < 2 * kP; ++q) {
    float v[2];
    rounded(q >> 1, v[0], v[1]);
    const float w = q & 1 ? v[1] : v[0], t = w * up;
    float n = fmaf(t, r, kMagic) - kMagic;
    const float off = fmaf(t, r, -n);
    if (fabsf(off) > 0.5f - kNear<kRot>) {
      // the codes below and above, and the border between them
      const float lo = off > 0.0f ? n : n - 1.0f;
      const Two e = mul({127.0f, 0.0f}, exact(q >> 1, q & 1, w, up));
      const Two border = mul({lo + 0.5f, 0.0f}, y);
      const bool even = ((int)lo & 1) == 0;
      n = less(e, border) || (!less(border, e) && even) ? lo : lo + 1.0f;
    }
    codes[lane + 32 * (q >> 1) + (q & 1) * kHalf] = (uint8_t)((int)n + 128);
  }
  if (lane == 0) *scale = fminf(amax / 127.0f, kMaxScale);
}

// Quantises one row of 8 values a lane (x[0..3] in the lower half, x[4..7] in the
// upper) and stores it, if `slot` says where. True: the row has to be taken by
// quantise_border_row (the same for every lane of the row, whatever rows share the
// warp).
//
// kTies: the values are bf16 as they came. With X and A the 8-bit significands of x
// and amax, a quotient t = 127 X 2^e / A lies on a border or at least t / (254 X),
// 1.5e-5 t, away from it. So t is rounded to a grid of its own size before its code
// is: p = 64 t, q = p - t rounded, p - q. The difference is exact and differs from t by
// q's rounding alone, at most half of a step of q, 2^-24 64 t = 3.8e-6 t; the borders
// (k + 1/2, k < 127) are on q's grid, and the f32 quotient of one, within 1.2e-7 t,
// goes to it (half a step is at least 1.9e-6 t), so that the sum with kMagic sees
// the tie. Ties are common in such rows: x = amax / 2, 63.5 codes, is in a third of
// normal rows of 128. Found by a comparison and a branch they took 11 us of 111.
template <int HD, bool kRot, bool kTies>
__device__ __forceinline__ bool quantise_row(const float (&x)[8], uint8_t* codes, float* scales,
                                             int64_t slot, int sub) {
  constexpr int kL = HD / 8;  // lanes of the row
  float amax = max_abs(x);
  bool odd = !(amax <= 1e30f);  // also NaN
#pragma unroll
  for (int o = kL / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
  odd |= amax > 0.0f && amax < 1e-30f;
  const float r = amax > 0.0f ? 127.0f / amax : 0.0f;
  float u[8];
  bool border = false;
  if constexpr (kTies) {
    const float r64 = r * 64.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float p = __fmul_rn(x[j], r64), q = fmaf(-x[j], r, p);
      u[j] = __fadd_rn(__fsub_rn(p, q), kMagic);
    }
  } else {
    float off[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      u[j] = fmaf(x[j], r, kMagic);
      off[j] = fmaf(x[j], r, kMagic - u[j]);  // distance to the code
    }
    border = max_abs(off) > 0.5f - kNear<kRot>;
  }
  const unsigned left = __ballot_sync(kAll, odd || border);
  const unsigned row = (kL == 32 ? kAll : (1u << (kL & 31)) - 1) << (threadIdx.x % 32 - sub);
  if (slot < 0) return false;
  if (left & row) return true;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = __byte_perm(__float_as_uint(u[4 * h]), __float_as_uint(u[4 * h + 1]), 0x0040);
    const uint32_t b = __byte_perm(__float_as_uint(u[4 * h + 2]), __float_as_uint(u[4 * h + 3]), 0x0040);
    *reinterpret_cast<uint32_t*>(codes + slot * HD + h * (HD / 2) + sub * 4) = __byte_perm(a, b, 0x5410);
  }
  if (sub == 0) scales[slot] = amax / 127.0f;
  return false;
}

// Twelve blocks an SM: what a block cannot hide of the two dependent loads before a
// row's store (position, then its rotation; lane, then its page), the others do.
// kTrace: with the step kernels' trace marks (0.4 us of a small call's 2.4).
template <typename T, int HD, bool kRot, bool kVec, bool kTrace>
__global__ void __launch_bounds__(kT, 12)
    k_kv_q8_append(KvQ8 c, const T* __restrict__ k, const T* __restrict__ v, int64_t k_stride,
                   int64_t v_stride, const int32_t* __restrict__ lanes,
                   const int32_t* __restrict__ positions, unsigned items,
                   const float* __restrict__ rc, const float* __restrict__ rs, int rope_len) {
  constexpr int kL = HD / 8, kHalf = HD / 2;
  __shared__ unsigned long long s_tr[kTrace ? 4 : 1];
  if constexpr (kTrace) TraceSmem::begin(s_tr, g_trace);
  pdl_wait();
  if constexpr (kTrace) TraceSmem::ready(s_tr);
  pdl_trigger();
  const int sub = threadIdx.x % kL;
  const unsigned at = (unsigned)(((uint64_t)blockIdx.x * kT + threadIdx.x) / kL);
  const unsigned item = min(at, items - 1);  // lanes past the end follow along and store nothing
  const unsigned i = c.by_head.div(item);
  const int g = (int)(item - i * c.Hkv);
  const T* kr = k + i * k_stride + (int64_t)g * HD;
  const T* vr = v + i * v_stride + (int64_t)g * HD;
  float x[8], y[8];
  load4<kVec>(kr + sub * 4, x);
  load4<kVec>(kr + sub * 4 + kHalf, x + 4);
  load4<kVec>(vr + sub * 4, y);
  load4<kVec>(vr + sub * 4 + kHalf, y + 4);
  const int pos = positions[i];
  int64_t slot = at < items ? q8::slot_of(c, lanes[i], pos, g) : -1;
  int64_t angles = 0;
  if constexpr (kRot) {
    if (pos < 0 || pos >= rope_len)
      slot = -1;
    else
      angles = (int64_t)pos * kHalf;
    float co[4], si[4];
    load4<kVec>(rc + angles + sub * 4, co);
    load4<kVec>(rs + angles + sub * 4, si);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x0 = x[j], x1 = x[j + 4];
      rope_pair(x0, x1, co[j], si[j], x[j], x[j + 4]);
    }
  }
  const bool k_left = quantise_row<HD, kRot, !kRot && sizeof(T) == 2>(x, c.k, c.ks, slot, sub);
  const bool v_left = quantise_row<HD, false, sizeof(T) == 2>(y, c.v, c.vs, slot, sub);
  // the warp takes the rows that are left one by one
  const int lane = threadIdx.x & 31;
  for (unsigned m = __ballot_sync(kAll, sub == 0 && (k_left || v_left)); m; m &= m - 1) {
    const int src = __ffs(m) - 1;
    const bool do_k = __shfl_sync(kAll, k_left, src), do_v = __shfl_sync(kAll, v_left, src);
    const int64_t to = __shfl_sync(kAll, slot, src), an = __shfl_sync(kAll, angles, src);
    const int64_t ko = __shfl_sync(kAll, (int64_t)(kr - k), src);
    const int64_t vo = __shfl_sync(kAll, (int64_t)(vr - v), src);
    if (do_k)
      quantise_border_row<T, HD, kRot>(k + ko, rc + an, rs + an, c.k + to * HD, c.ks + to, lane);
    if (do_v)
      quantise_border_row<T, HD, false>(v + vo, nullptr, nullptr, c.v + to * HD, c.vs + to, lane);
  }
  if constexpr (kTrace) TraceSmem::end(s_tr, TR_KV_Q8_APPEND);
}

__device__ __forceinline__ void values4(uint32_t w, float s, float x[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)  // 2^23 + byte, less 2^23 + 128
    x[j] = (__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440 + j)) - 8388736.0f) * s;
}

template <typename T, int HD, bool kVec>
__global__ void __launch_bounds__(kT)
    k_kv_q8_read(KvQ8 c, const int32_t* __restrict__ lanes, const int32_t* __restrict__ positions,
                 unsigned items, T* __restrict__ k_out, T* __restrict__ v_out, int64_t k_stride,
                 int64_t v_stride) {
  constexpr int kL = HD / 8, kHalf = HD / 2;
  pdl_wait();
  pdl_trigger();
  const int sub = threadIdx.x % kL;
  const unsigned item = (unsigned)(((uint64_t)blockIdx.x * kT + threadIdx.x) / kL);
  if (item >= items) return;
  const unsigned i = c.by_head.div(item);
  const int g = (int)(item - i * c.Hkv);
  const int64_t slot = q8::slot_of(c, lanes[i], positions[i], g);
  // a token of no slot reads as zeros: scale 0
  uint32_t kw[2] = {0, 0}, vw[2] = {0, 0};
  float ks = 0.0f, vs = 0.0f;
  if (slot >= 0) {
    const int64_t p = slot * HD + sub * 4;
    if (k_out) {
      kw[0] = *reinterpret_cast<const uint32_t*>(c.k + p);
      kw[1] = *reinterpret_cast<const uint32_t*>(c.k + p + kHalf);
      ks = c.ks[slot];
    }
    if (v_out) {
      vw[0] = *reinterpret_cast<const uint32_t*>(c.v + p);
      vw[1] = *reinterpret_cast<const uint32_t*>(c.v + p + kHalf);
      vs = c.vs[slot];
    }
  }
  float x[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (k_out) {
      values4(kw[h], ks, x);
      store4<kVec>(k_out + i * k_stride + (int64_t)g * HD + sub * 4 + h * kHalf, x);
    }
    if (v_out) {
      values4(vw[h], vs, x);
      store4<kVec>(v_out + i * v_stride + (int64_t)g * HD + sub * 4 + h * kHalf, x);
    }
  }
}

__device__ __forceinline__ uint64_t mix64(uint64_t z) {  // splitmix64 finaliser
  z += 0x9E3779B97F4A7C15ull;
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

// Fills whole pages of every layer, K and V, with codes uniform in -127 .. 127 under
// scales sqrt(3) / 127 (unit variance), from (seed, word index).
__global__ void k_fill_random_kv_q8(KvQ8 c, int L, int64_t layer_rows,
                                    const int32_t* __restrict__ pages, int n_pages, uint64_t seed) {
  const int64_t page_rows = (int64_t)c.Hkv * c.page_size, row_words = c.hd / 4;
  const int64_t per_layer = n_pages * page_rows * row_words;
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < L * per_layer;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int64_t l = i / per_layer, rest = i - l * per_layer;
    const int64_t r = rest / row_words, w = rest - r * row_words;
    const int64_t row = l * layer_rows + pages[r / page_rows] * page_rows + r % page_rows;
    const int64_t word = row * row_words + w;
    uint32_t out[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t u = (uint32_t)(mix64(seed ^ (uint64_t)(8 * word + j)) >> 40);  // 24 bits
      out[j / 4] |= (1u + (uint32_t)(((uint64_t)u * 255u) >> 24)) << (8 * (j % 4));
    }
    reinterpret_cast<uint32_t*>(c.k)[word] = out[0];
    reinterpret_cast<uint32_t*>(c.v)[word] = out[1];
    if (w == 0) c.ks[row] = c.vs[row] = 1.7320508f / 127.0f;
  }
}

// k_kv_relocate (k_misc.cu) for an 8-bit cache: rows [q_begin, q_end) of one lane into
// the pages of dst_pt, row q from row q (q < a) or q + delta of src_pt's pages. A row
// that keeps its place, and every value row, moves as it is stored; a key that moves
// down by delta is turned back by delta positions and quantised anew. One block per
// (layer, KV head, K|V) walks its rows in ascending batches, a warp a row; a batch is
// read whole before any of it is written.
constexpr int kRelocWarps = 8;
template <int HD>
__global__ void __launch_bounds__(32 * kRelocWarps)
    k_kv_q8_relocate(KvQ8 c, int64_t layer_rows, const int32_t* __restrict__ src_pt,
                     const int32_t* __restrict__ dst_pt, int q_begin, int q_end, int a, int delta,
                     const float* __restrict__ rc, const float* __restrict__ rs) {
  constexpr int kHalf = HD / 2, kP = HD / 64;
  const bool values = blockIdx.x & 1;
  const int g = (int)(blockIdx.x >> 1) % c.Hkv;
  const int64_t base = (int64_t)((blockIdx.x >> 1) / c.Hkv) * layer_rows;
  uint8_t* codes = values ? c.v : c.k;
  float* scales = values ? c.vs : c.ks;
  auto row_of = [&](const int32_t* pt, int t) {
    const int pi = (int)c.by_page.div(t);
    return base + ((int64_t)pt[pi] * c.Hkv + g) * c.page_size + (t - pi * c.page_size);
  };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r0 = q_begin; r0 < q_end; r0 += kRelocWarps) {
    const int q = r0 + warp;
    uint8_t lo[kP] = {}, hi[kP] = {};
    float s = 0.0f;
    if (q < q_end) {
      const int64_t from = row_of(src_pt, q < a ? q : q + delta);
      s = scales[from];
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        lo[p] = codes[from * HD + lane + 32 * p];
        hi[p] = codes[from * HD + kHalf + lane + 32 * p];
      }
      if (!values && q >= a && delta > 0) {  // the same for every lane of the warp
        float y0[kP], y1[kP], amax = 0.0f;
#pragma unroll
        for (int p = 0; p < kP; ++p) {
          const int64_t at = (int64_t)delta * kHalf + lane + 32 * p;
          rope_pair((float)((int)lo[p] - 128) * s, (float)((int)hi[p] - 128) * s, rc[at], -rs[at],
                    y0[p], y1[p]);
          y0[p] = storable(y0[p]), y1[p] = storable(y1[p]);
          amax = fmaxf(amax, fmaxf(fabsf(y0[p]), fabsf(y1[p])));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
#pragma unroll
        for (int p = 0; p < kP; ++p) {
          lo[p] = (uint8_t)(128 + (amax > 0.0f ? (int)rintf(y0[p] / amax * 127.0f) : 0));
          hi[p] = (uint8_t)(128 + (amax > 0.0f ? (int)rintf(y1[p] / amax * 127.0f) : 0));
        }
        s = fminf(amax / 127.0f, kMaxScale);
      }
    }
    __syncthreads();
    if (q < q_end) {
      const int64_t to = row_of(dst_pt, q);
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        codes[to * HD + lane + 32 * p] = lo[p];
        codes[to * HD + kHalf + lane + 32 * p] = hi[p];
      }
      if (lane == 0) scales[to] = s;
    }
    __syncthreads();
  }
}

unsigned blocks(unsigned items, int hd) {
  return (unsigned)(((uint64_t)items * (hd / 8) + kT - 1) / kT);
}

// Rows whose groups of four elements are aligned (16 bytes of f32, 8 of bf16).
bool rows_aligned(const void* p, int64_t stride, size_t es) {
  return reinterpret_cast<uintptr_t>(p) % (4 * es) == 0 && stride % 4 == 0;
}

template <typename T, int HD, bool kTrace>
Launched append_hd(const KvQ8& c, const void* k, const void* v, int64_t k_stride,
                   int64_t v_stride, const int32_t* lanes, const int32_t* positions, int n,
                   const float* rc, const float* rs, int rope_len, cudaStream_t s) {
  const unsigned items = (unsigned)((int64_t)n * c.Hkv);
  const bool vec = rows_aligned(k, k_stride, sizeof(T)) && rows_aligned(v, v_stride, sizeof(T)) &&
                   rows_aligned(rc, 4, 4) && rows_aligned(rs, 4, 4);
  auto kern = rc ? (vec ? k_kv_q8_append<T, HD, true, true, kTrace>
                        : k_kv_q8_append<T, HD, true, false, kTrace>)
                 : (vec ? k_kv_q8_append<T, HD, false, true, kTrace>
                        : k_kv_q8_append<T, HD, false, false, kTrace>);
  Launched l;
  l.add(launch_k(kern, dim3(blocks(items, HD)), kT, 0, s, c, static_cast<const T*>(k),
                 static_cast<const T*>(v), k_stride, v_stride, lanes, positions, items, rc, rs,
                 rope_len));
  return l;
}

template <int HD, typename... A>
Launched append_types(const KvQ8& c, int x_type, bool traced, A... a) {
  if (x_type == X_BF16) return append_hd<__nv_bfloat16, HD, false>(c, a...);
  return traced ? append_hd<float, HD, true>(c, a...) : append_hd<float, HD, false>(c, a...);
}

template <typename T, int HD>
Launched read_hd(const KvQ8& c, const int32_t* lanes, const int32_t* positions, int n, void* k_out,
                 void* v_out, int64_t k_stride, int64_t v_stride, cudaStream_t s) {
  const unsigned items = (unsigned)((int64_t)n * c.Hkv);
  const bool vec = (!k_out || rows_aligned(k_out, k_stride, sizeof(T))) &&
                   (!v_out || rows_aligned(v_out, v_stride, sizeof(T)));
  auto kern = vec ? k_kv_q8_read<T, HD, true> : k_kv_q8_read<T, HD, false>;
  Launched l;
  l.add(launch_k(kern, dim3(blocks(items, HD)), kT, 0, s, c, lanes, positions, items,
                 static_cast<T*>(k_out), static_cast<T*>(v_out), k_stride, v_stride));
  return l;
}

}  // namespace

bool kv_q8_supports(int hd) { return hd == 64 || hd == 128 || hd == 256; }

Launched launch_kv_q8_append(const KvQ8& c, const void* k, const void* v, int64_t k_stride,
                             int64_t v_stride, int x_type, bool traced, const int32_t* lanes,
                             const int32_t* positions, int n, const float* rc, const float* rs,
                             int rope_len, cudaStream_t s) {
  if (n <= 0) return {};
  auto go = [&](auto hd) {
    return append_types<decltype(hd)::value>(c, x_type, traced, k, v, k_stride, v_stride, lanes,
                                             positions, n, rc, rs, rope_len, s);
  };
  return c.hd == 64    ? go(std::integral_constant<int, 64>())
         : c.hd == 128 ? go(std::integral_constant<int, 128>())
         : c.hd == 256 ? go(std::integral_constant<int, 256>())
                       : Launched{};
}

Launched launch_kv_q8_read(const KvQ8& c, const int32_t* lanes, const int32_t* positions, int n,
                           void* k_out, void* v_out, int64_t k_stride, int64_t v_stride,
                           int x_type, cudaStream_t s) {
  if (n <= 0) return {};
  auto go = [&](auto hd) {
    constexpr int HD = decltype(hd)::value;
    return x_type == X_BF16 ? read_hd<__nv_bfloat16, HD>(c, lanes, positions, n, k_out, v_out,
                                                         k_stride, v_stride, s)
                            : read_hd<float, HD>(c, lanes, positions, n, k_out, v_out, k_stride,
                                                 v_stride, s);
  };
  return c.hd == 64    ? go(std::integral_constant<int, 64>())
         : c.hd == 128 ? go(std::integral_constant<int, 128>())
         : c.hd == 256 ? go(std::integral_constant<int, 256>())
                       : Launched{};
}

int launch_fill_random_kv_q8(const KvQ8& c, int L, int64_t layer_rows, const int32_t* pages,
                             int n_pages, uint64_t seed, cudaStream_t s) {
  if (n_pages <= 0) return 0;
  k_fill_random_kv_q8<<<1216, 256, 0, s>>>(c, L, layer_rows, pages, n_pages, seed);
  return 1;
}

int launch_kv_q8_relocate(const KvQ8& c, int L, int64_t layer_rows, const int32_t* src_pt,
                          const int32_t* dst_pt, int q_begin, int q_end, int a, int delta,
                          const float* rc, const float* rs, cudaStream_t s) {
  if (q_end <= q_begin) return 0;
  auto kern = c.hd == 64    ? k_kv_q8_relocate<64>
              : c.hd == 128 ? k_kv_q8_relocate<128>
                            : k_kv_q8_relocate<256>;
  kern<<<(unsigned)L * c.Hkv * 2, 32 * kRelocWarps, 0, s>>>(c, layer_rows, src_pt, dst_pt, q_begin,
                                                            q_end, a, delta, rc, rs);
  return 1;
}

}  // namespace fsk
