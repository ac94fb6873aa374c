// Quantised writes into the 8-bit paged KV cache, and reads back out of it.
//
// A row x of hd values (one token, one KV head; keys after their rotation)
// is stored as scale = amax / 127 and codes round(x * 127 / amax), ties to
// even, amax the largest magnitude; a value stands for code * scale.

#include <float.h>

#include "kv_q8.cuh"

namespace fsk {
namespace {

constexpr int kWarps = 8;  // (row, head) pairs per block, one warp each

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// What a cache row can hold: NaN becomes 0, infinities the largest finite f32.
__device__ __forceinline__ float storable(float x) {
  return x != x ? 0.0f : fminf(fmaxf(x, -FLT_MAX), FLT_MAX);
}
__device__ __forceinline__ double storable(double x) {
  return x != x ? 0.0 : fmin(fmax(x, -(double)FLT_MAX), (double)FLT_MAX);
}

// One warp quantises one row: lane l holds elements l * E .. l * E + E - 1 of
// the lower half (x[0..E)) and of the upper half (x[E..2E)), E = HD / 64.
//
// The quotient in f32 is off by at most 1.3e-4 of a step: the factor 127 / amax
// and the product round by 2^-24 each of at most 127 (1.5e-5 together), a
// rotated x by (2 sqrt 2 + 1) 2^-24 amax (2.9e-5 steps), and amax likewise,
// all with room. Where a quotient comes that near to the border of two codes
// the warp takes the row again in 64 bits (`again` gives the exact elements):
// about one row in thirty at HD = 128.
template <int HD, typename Again>
__device__ __forceinline__ void quantise_row(const float (&x)[HD / 32], Again again,
                                             uint8_t* __restrict__ codes,
                                             float* __restrict__ scale, int lane) {
  constexpr int N = HD / 32, E = N / 2;
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) amax = fmaxf(amax, fabsf(x[j]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float r = 127.0f / amax;
  int c[N];
  bool border = amax < 1e-30f;  // 127 / amax may not be finite
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float t = x[j] * r, n = rintf(t);
    border |= fabsf(t - n) > 0.5f - 1.3e-4f;
    c[j] = (int)n;
  }
  float s = amax / 127.0f;
  if (__any_sync(0xffffffffu, border)) {
    double y[N], ymax = 0.0;
    again(y);
#pragma unroll
    for (int j = 0; j < N; ++j) ymax = fmax(ymax, fabs(y[j]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ymax = fmax(ymax, __shfl_xor_sync(0xffffffffu, ymax, o));
#pragma unroll
    for (int j = 0; j < N; ++j) c[j] = ymax > 0.0 ? (int)rint(y[j] * 127.0 / ymax) : 0;
    s = (float)(ymax / 127.0);
  }
#pragma unroll
  for (int j = 0; j < N; ++j)
    codes[(j / E) * (HD / 2) + lane * E + j % E] = (uint8_t)(c[j] + 128);
  if (lane == 0) *scale = s;
}

template <typename T, int HD>
__global__ void __launch_bounds__(32 * kWarps)
    k_kv_q8_append(KvQ8 c, const T* __restrict__ k, const T* __restrict__ v, int64_t k_stride,
                   int64_t v_stride, const int32_t* __restrict__ lanes,
                   const int32_t* __restrict__ positions, int n, const float* __restrict__ rc,
                   const float* __restrict__ rs, int rope_len) {
  constexpr int N = HD / 32, E = N / 2, kHalf = HD / 2;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= (int64_t)n * c.Hkv) return;
  const int i = (int)(item / c.Hkv), g = (int)(item - (int64_t)i * c.Hkv);
  const int pos = positions[i];
  const int64_t slot = q8::slot_of(c, lanes[i], pos, g);
  if (slot < 0 || (rc && pos >= rope_len)) return;  // a row of no token: nothing is written
  const T* kr = k + i * k_stride + (int64_t)g * HD;
  const T* vr = v + i * v_stride + (int64_t)g * HD;
  float kx[N], vx[N], co[E], si[E];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int at = (j / E) * kHalf + lane * E + j % E;
    kx[j] = ld1(kr + at);
    vx[j] = storable(ld1(vr + at));
  }
#pragma unroll
  for (int j = 0; j < E; ++j) {
    co[j] = rc ? rc[(int64_t)pos * kHalf + lane * E + j] : 1.0f;
    si[j] = rc ? rs[(int64_t)pos * kHalf + lane * E + j] : 0.0f;
  }
  float y[N];
#pragma unroll
  for (int j = 0; j < E; ++j) {
    rope_pair(kx[j], kx[j + E], co[j], si[j], y[j], y[j + E]);
    y[j] = storable(rc ? y[j] : kx[j]);
    y[j + E] = storable(rc ? y[j + E] : kx[j + E]);
  }
  quantise_row<HD>(
      y,
      [&](double (&d)[N]) {
#pragma unroll
        for (int j = 0; j < E; ++j) {
          const double a = kx[j], b = kx[j + E], cc = co[j], ss = si[j];
          d[j] = storable(rc ? a * cc - b * ss : a);
          d[j + E] = storable(rc ? b * cc + a * ss : b);
        }
      },
      c.k + slot * HD, c.ks + slot, lane);
  quantise_row<HD>(
      vx,
      [&](double (&d)[N]) {
#pragma unroll
        for (int j = 0; j < N; ++j) d[j] = vx[j];
      },
      c.v + slot * HD, c.vs + slot, lane);
}

template <typename T, int HD>
__global__ void __launch_bounds__(32 * kWarps)
    k_kv_q8_read(KvQ8 c, const int32_t* __restrict__ lanes,
                 const int32_t* __restrict__ positions, int n, T* __restrict__ k_out,
                 T* __restrict__ v_out, int64_t k_stride, int64_t v_stride) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= (int64_t)n * c.Hkv) return;
  const int i = (int)(item / c.Hkv), g = (int)(item - (int64_t)i * c.Hkv);
  const int64_t slot = q8::slot_of(c, lanes[i], positions[i], g);
  for (int d = lane; d < HD; d += 32) {
    if (k_out)
      st1(k_out + i * k_stride + (int64_t)g * HD + d,
          slot < 0 ? 0.0f : (float)((int)c.k[slot * HD + d] - 128) * c.ks[slot]);
    if (v_out)
      st1(v_out + i * v_stride + (int64_t)g * HD + d,
          slot < 0 ? 0.0f : (float)((int)c.v[slot * HD + d] - 128) * c.vs[slot]);
  }
}

template <typename T, int HD>
void append_hd(const KvQ8& c, const void* k, const void* v, int64_t k_stride, int64_t v_stride,
               const int32_t* lanes, const int32_t* positions, int n, const float* rc,
               const float* rs, int rope_len, cudaStream_t s) {
  const int64_t items = (int64_t)n * c.Hkv;
  launch_k(k_kv_q8_append<T, HD>, dim3((unsigned)((items + kWarps - 1) / kWarps)), 32 * kWarps, 0,
           s, c, static_cast<const T*>(k), static_cast<const T*>(v), k_stride, v_stride, lanes,
           positions, n, rc, rs, rope_len);
}

template <typename T, int HD>
void read_hd(const KvQ8& c, const int32_t* lanes, const int32_t* positions, int n, void* k_out,
             void* v_out, int64_t k_stride, int64_t v_stride, cudaStream_t s) {
  const int64_t items = (int64_t)n * c.Hkv;
  launch_k(k_kv_q8_read<T, HD>, dim3((unsigned)((items + kWarps - 1) / kWarps)), 32 * kWarps, 0, s,
           c, lanes, positions, n, static_cast<T*>(k_out), static_cast<T*>(v_out), k_stride,
           v_stride);
}

}  // namespace

bool kv_q8_supports(int hd) { return hd == 64 || hd == 128 || hd == 256; }

#define FS_Q8_DISPATCH(fn, ...)                                                       \
  switch (c.hd) {                                                                     \
    case 64:                                                                          \
      x_type == X_BF16 ? fn<__nv_bfloat16, 64>(__VA_ARGS__) : fn<float, 64>(__VA_ARGS__);   \
      return 1;                                                                       \
    case 128:                                                                         \
      x_type == X_BF16 ? fn<__nv_bfloat16, 128>(__VA_ARGS__) : fn<float, 128>(__VA_ARGS__); \
      return 1;                                                                       \
    case 256:                                                                         \
      x_type == X_BF16 ? fn<__nv_bfloat16, 256>(__VA_ARGS__) : fn<float, 256>(__VA_ARGS__); \
      return 1;                                                                       \
    default:                                                                          \
      return 0;                                                                       \
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
