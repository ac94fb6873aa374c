// Quantised writes into the 8-bit paged KV cache, and reads back out of it.
//
// A row x of hd values (one token, one KV head; keys after their rotation)
// is stored as scale = amax / 127 and codes round(x * 127 / amax), ties to
// even, amax the largest magnitude; a value stands for code * scale.
//
// Both directions are bound by HBM when there are many rows. hd / 8 lanes share a
// row, each with four values of its lower and four of its upper half (what a
// rotation pairs), so that the loads and stores of a warp are whole sectors of
// consecutive rows, and every lane has its key and its value row in flight
// together. Rounding to a code is one fused multiply-add: x * r + 1.5 * 2^23 + 128
// has the byte code + 128 in its last bits.

#include <float.h>

#include "kv_q8.cuh"
#include "two_f32.cuh"

namespace fsk {
namespace {

using namespace two;

constexpr int kT = 256;
constexpr unsigned kAll = 0xffffffffu;

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
template <bool kVec>
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float x[4]) {
  if constexpr (kVec) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) p[j] = __float2bfloat16_rn(x[j]);
  }
}

// What a cache row can hold: NaN becomes 0, infinities the largest finite f32.
__device__ __forceinline__ float storable(float x) {
  return x != x ? 0.0f : fminf(fmaxf(x, -FLT_MAX), FLT_MAX);
}

// Quantises one row of 8 values a lane (x[0..3] in the lower half, x[4..7] in the
// upper) and stores it, if `slot` says where.
//
// A quotient in f32 is off by at most kNear of a step: the factor 127 / amax and
// the product round by 2^-24 of at most 127 each, 1.6e-5 together; of a rotated
// key x is off by (1 + sqrt 2) 2^-24 amax, two rounded products and their sum,
// 1.9e-5 of a step, and amax likewise. A quotient that comes so near to the border
// of two codes (one row of 128 in 200 for values, in 65 for rotated keys) is
// decided by comparing 127 x with the border times amax as two-f32 numbers:
// exactly for values that were not rotated, to 2^-44 for others (exact(j, up) is
// element j times a power of two so). In f64 these rows alone took four fifths
// of the kernel (65536 rows of 8 heads of 128: 473 us).
template <int HD, bool kRot, typename Exact>
__device__ __forceinline__ void quantise_row(const float (&x)[8], Exact exact, uint8_t* codes,
                                             float* scales, int64_t slot, int sub) {
  constexpr int kL = HD / 8;  // lanes of the row
  constexpr float kNear = kRot ? 6e-5f : 2e-5f;
  constexpr float kMagic = 12582912.0f + 128.0f;
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
#pragma unroll
  for (int o = kL / 2; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, o));
  // into the range where quotients and products neither overflow nor vanish
  const float up = amax < 1e-30f ? 0x1p96f : amax > 1e30f ? 0x1p-96f : 1.0f;
  const float top = amax * up, r = top > 0.0f ? 127.0f / top : 0.0f;
  float u[8], off = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float xs = x[j] * up;
    u[j] = fmaf(xs, r, kMagic);
    off = fmaxf(off, fabsf(fmaf(xs, r, kMagic - u[j])));  // distance to the code
  }
  // by row, not by warp: a row's bits do not depend on the rows beside it
  const unsigned near = __ballot_sync(kAll, off > 0.5f - kNear);
  const unsigned row = (kL == 32 ? kAll : (1u << (kL & 31)) - 1) << (threadIdx.x % 32 - sub);
  if (near & row) {
    Two y = {top, 0.0f};
    if constexpr (kRot) {  // the largest magnitude: of the lanes that hold it in f32
      y = {0.0f, 0.0f};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (fabsf(x[j]) >= amax * (1.0f - 0x1p-20f)) {
          Two e = exact(j, up);
          if (e.h < 0.0f) e = {-e.h, -e.l};
          if (less(y, e)) y = e;
        }
#pragma unroll
      for (int o = kL / 2; o > 0; o >>= 1) {
        const Two e = {__shfl_xor_sync(row, y.h, o), __shfl_xor_sync(row, y.l, o)};
        if (less(y, e)) y = e;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float n = u[j] - kMagic, d = fmaf(x[j] * up, r, -n);
      if (fabsf(d) > 0.5f - kNear) {
        // the codes below and above, and the border between them
        const float lo = d > 0.0f ? n : n - 1.0f;
        const Two e = mul({127.0f, 0.0f}, exact(j, up)), border = mul({lo + 0.5f, 0.0f}, y);
        const bool even = ((int)lo & 1) == 0;
        const bool below = less(e, border) || (!less(border, e) && even);
        u[j] = kMagic + (below ? lo : lo + 1.0f);
      }
    }
  }
  if (slot < 0) return;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = __byte_perm(__float_as_uint(u[4 * h]), __float_as_uint(u[4 * h + 1]), 0x0040);
    const uint32_t b = __byte_perm(__float_as_uint(u[4 * h + 2]), __float_as_uint(u[4 * h + 3]), 0x0040);
    *reinterpret_cast<uint32_t*>(codes + slot * HD + h * (HD / 2) + sub * 4) = __byte_perm(a, b, 0x5410);
  }
  if (sub == 0) scales[slot] = amax / 127.0f;
}

template <typename T, int HD, bool kRot, bool kVec>
__global__ void __launch_bounds__(kT)
    k_kv_q8_append(KvQ8 c, const T* __restrict__ k, const T* __restrict__ v, int64_t k_stride,
                   int64_t v_stride, const int32_t* __restrict__ lanes,
                   const int32_t* __restrict__ positions, unsigned items,
                   const float* __restrict__ rc, const float* __restrict__ rs, int rope_len) {
  constexpr int kL = HD / 8, kHalf = HD / 2;
  pdl_wait();
  pdl_trigger();
  const int sub = threadIdx.x % kL;
  const unsigned at = (unsigned)(((uint64_t)blockIdx.x * kT + threadIdx.x) / kL);
  const unsigned item = min(at, items - 1);  // lanes past the end follow along and store nothing
  const unsigned i = item / (unsigned)c.Hkv;
  const int g = (int)(item - i * c.Hkv);
  const T* kr = k + i * k_stride + (int64_t)g * HD + sub * 4;
  const T* vr = v + i * v_stride + (int64_t)g * HD + sub * 4;
  float kx[8], vx[8];
  load4<kVec>(kr, kx);
  load4<kVec>(kr + kHalf, kx + 4);
  load4<kVec>(vr, vx);
  load4<kVec>(vr + kHalf, vx + 4);
  const int pos = positions[i];
  int64_t slot = at < items ? q8::slot_of(c, lanes[i], pos, g) : -1;
  float y[8], co[4] = {}, si[4] = {};
  if constexpr (kRot) {
    const bool in = pos >= 0 && pos < rope_len;
    if (!in) slot = -1;
    const int64_t p = in ? (int64_t)pos * kHalf + sub * 4 : 0;
    load4<kVec>(rc + p, co);
    load4<kVec>(rs + p, si);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      rope_pair(kx[j], kx[j + 4], co[j], si[j], y[j], y[j + 4]);
      y[j] = storable(y[j]);
      y[j + 4] = storable(y[j + 4]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = storable(kx[j]);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) vx[j] = storable(vx[j]);
  quantise_row<HD, kRot>(
      y,
      [&](int j, float up) -> Two {
        if (!kRot || fabsf(y[j]) >= FLT_MAX) return {y[j] * up, 0.0f};
        const float a0 = kx[j & 3] * up, b0 = kx[(j & 3) + 4] * up, cc = co[j & 3], ss = si[j & 3];
        return j < 4 ? add(two_prod(a0, cc), two_prod(b0, -ss))
                     : add(two_prod(b0, cc), two_prod(a0, ss));
      },
      c.k, c.ks, slot, sub);
  quantise_row<HD, false>(
      vx, [&](int j, float up) -> Two { return {vx[j] * up, 0.0f}; }, c.v, c.vs, slot, sub);
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
  const unsigned i = item / (unsigned)c.Hkv;
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

unsigned blocks(unsigned items, int hd) {
  return (unsigned)(((uint64_t)items * (hd / 8) + kT - 1) / kT);
}

// Rows whose groups of four elements are aligned (16 bytes of f32, 8 of bf16).
bool rows_aligned(const void* p, int64_t stride, size_t es) {
  return reinterpret_cast<uintptr_t>(p) % (4 * es) == 0 && stride % 4 == 0;
}

template <typename T, int HD>
void append_hd(const KvQ8& c, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
               const int32_t* lanes, const int32_t* positions, int n, const float* rc,
               const float* rs, int rope_len, cudaStream_t s) {
  const unsigned items = (unsigned)((int64_t)n * c.Hkv);
  const bool vec = rows_aligned(k, k_stride, sizeof(T)) && rows_aligned(v, v_stride, sizeof(T)) &&
                   rows_aligned(rc, 4, 4) && rows_aligned(rs, 4, 4);
  auto kern = rc ? (vec ? k_kv_q8_append<T, HD, true, true> : k_kv_q8_append<T, HD, true, false>)
                 : (vec ? k_kv_q8_append<T, HD, false, true> : k_kv_q8_append<T, HD, false, false>);
  launch_k(kern, dim3(blocks(items, HD)), kT, 0, s, c, static_cast<const T*>(k),
           static_cast<const T*>(v), k_stride, v_stride, lanes, positions, items, rc, rs, rope_len);
}

template <typename T, int HD>
void read_hd(const KvQ8& c, const int32_t* lanes, const int32_t* positions, int n, void* k_out,
             void* v_out, int64_t k_stride, int64_t v_stride, cudaStream_t s) {
  const unsigned items = (unsigned)((int64_t)n * c.Hkv);
  const bool vec = (!k_out || rows_aligned(k_out, k_stride, sizeof(T))) &&
                   (!v_out || rows_aligned(v_out, v_stride, sizeof(T)));
  auto kern = vec ? k_kv_q8_read<T, HD, true> : k_kv_q8_read<T, HD, false>;
  launch_k(kern, dim3(blocks(items, HD)), kT, 0, s, c, lanes, positions, items,
           static_cast<T*>(k_out), static_cast<T*>(v_out), k_stride, v_stride);
}

}  // namespace

bool kv_q8_supports(int hd) { return hd == 64 || hd == 128 || hd == 256; }

#define FS_Q8_DISPATCH(fn, ...)                                                             \
  switch (c.hd) {                                                                           \
    case 64:                                                                                \
      x_type == X_BF16 ? fn<__nv_bfloat16, 64>(__VA_ARGS__) : fn<float, 64>(__VA_ARGS__);   \
      return 1;                                                                             \
    case 128:                                                                               \
      x_type == X_BF16 ? fn<__nv_bfloat16, 128>(__VA_ARGS__) : fn<float, 128>(__VA_ARGS__); \
      return 1;                                                                             \
    case 256:                                                                               \
      x_type == X_BF16 ? fn<__nv_bfloat16, 256>(__VA_ARGS__) : fn<float, 256>(__VA_ARGS__); \
      return 1;                                                                             \
    default:                                                                                \
      return 0;                                                                             \
  }

int launch_kv_q8_append(const KvQ8& c, const void* k, const void* v, int64_t k_stride,
                        int64_t v_stride, int x_type, const int32_t* lanes,
                        const int32_t* positions, int n, const float* rc, const float* rs,
                        int rope_len, cudaStream_t s) {
  if (n <= 0) return 0;
  FS_Q8_DISPATCH(append_hd, c, k, v, k_stride, v_stride, lanes, positions, n, rc, rs, rope_len, s)
}

int launch_kv_q8_read(const KvQ8& c, const int32_t* lanes, const int32_t* positions, int n,
                      void* k_out, void* v_out, int64_t k_stride, int64_t v_stride, int x_type,
                      cudaStream_t s) {
  if (n <= 0) return 0;
  FS_Q8_DISPATCH(read_hd, c, lanes, positions, n, k_out, v_out, k_stride, v_stride, s)
}

}  // namespace fsk
