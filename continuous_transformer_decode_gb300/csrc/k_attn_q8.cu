// Attention of one new token a row over the 8-bit paged KV cache, split over
// the cache's length and joined.
//
//   o_h = sum_t p_t v_t,  p = softmax_t(scale * q_h . k_t),  t < length
//
// with k_t = ks_t * code, v_t = vs_t * code. One block takes a split of one
// (row, KV head): its warps take positions in turn, each with the running
// maximum and sum of its own softmax, and are joined in warp order; the
// splits of a row, in f32, by a second kernel in split order.

#include <math_constants.h>

#include <algorithm>

#include "kv_q8.cuh"

namespace fsk {
namespace {

constexpr int kWarps = 4;
constexpr int kT = 32 * kWarps;
constexpr int kG = 8;  // query heads per KV head at most

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ int row_len(const AttnQ8& a, int i) {
  return min(min(max(a.lens[i], 0), a.max_len), a.kv.max_pages * a.kv.page_size);
}

template <typename QT, typename OT, int HD>
__global__ void __launch_bounds__(kT) k_attn_q8(AttnQ8 a) {
  constexpr int N = HD / 32;
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int H = a.H, G = H / a.kv.Hkv;
  const int len = row_len(a, b);
  const int start = s * a.split_len, end = min(len, start + a.split_len);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  OT* orow = static_cast<OT*>(a.out) + b * a.out_stride + (int64_t)g * G * HD;
  if (len == 0 && s == 0)
    for (int i = tid; i < G * HD; i += kT) st1(orow + i, 0.0f);
  if (start >= end) return;
  __shared__ float qs[kG][HD], wo[kWarps][kG][HD], wm[kWarps][kG], wl[kWarps][kG];
  const QT* qr = static_cast<const QT*>(a.q) + b * a.q_stride + (int64_t)g * G * HD;
  for (int i = tid; i < G * HD / 2; i += kT) {
    const int h = i / (HD / 2), j = i % (HD / 2);
    float x0 = ld1(qr + h * HD + j), x1 = ld1(qr + h * HD + j + HD / 2);
    if (a.rc) {
      const int64_t at = (int64_t)(len - 1) * (HD / 2) + j;
      float y0, y1;
      rope_pair(x0, x1, a.rc[at], a.rs[at], y0, y1);
      x0 = y0;
      x1 = y1;
    }
    qs[h][j] = x0 * a.scale;
    qs[h][j + HD / 2] = x1 * a.scale;
  }
  __syncthreads();
  float m[kG], l[kG], o[kG][N];
#pragma unroll
  for (int h = 0; h < kG; ++h) {
    m[h] = -CUDART_INF_F;
    l[h] = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) o[h][j] = 0.0f;
  }
  for (int t = start + warp; t < end; t += kWarps) {
    const int64_t slot = q8::slot_of(a.kv, a.lanes[b], t, g);
    if (slot < 0) continue;
    float k[N], v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      k[j] = (float)((int)a.kv.k[slot * HD + lane + 32 * j] - 128);
      v[j] = (float)((int)a.kv.v[slot * HD + lane + 32 * j] - 128);
    }
    const float ks = a.kv.ks[slot], vs = a.kv.vs[slot];
#pragma unroll
    for (int h = 0; h < kG; ++h) {
      if (h >= G) break;
      float z = 0.0f;
#pragma unroll
      for (int j = 0; j < N; ++j) z = fmaf(qs[h][lane + 32 * j], k[j], z);
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) z += __shfl_xor_sync(0xffffffffu, z, w);
      z *= ks;
      const float mn = fmaxf(m[h], z);
      const float alpha = m[h] == -CUDART_INF_F ? 0.0f : expf(m[h] - mn);
      const float p = expf(z - mn);
      m[h] = mn;
      l[h] = l[h] * alpha + p;
#pragma unroll
      for (int j = 0; j < N; ++j) o[h][j] = o[h][j] * alpha + p * vs * v[j];
    }
  }
#pragma unroll
  for (int h = 0; h < kG; ++h) {
    if (lane == 0) {
      wm[warp][h] = m[h];
      wl[warp][h] = l[h];
    }
#pragma unroll
    for (int j = 0; j < N; ++j) wo[warp][h][lane + 32 * j] = o[h][j];
  }
  __syncthreads();
  const int64_t base = ((int64_t)b * a.n_splits + s) * H + g * G;
  for (int i = tid; i < G * HD; i += kT) {
    const int h = i / HD, d = i % HD;
    float M = -CUDART_INF_F, L = 0.0f, A = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w][h]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float sc = wm[w][h] == -CUDART_INF_F ? 0.0f : expf(wm[w][h] - M);
      L = fmaf(wl[w][h], sc, L);
      A = fmaf(wo[w][h][d], sc, A);
    }
    if (len <= a.split_len) {
      st1(orow + i, L > 0.0f ? A / L : 0.0f);
    } else {
      a.part_acc[base * HD + i] = A;
      if (d == 0) {
        a.part_ml[2 * (base + h)] = M;
        a.part_ml[2 * (base + h) + 1] = L;
      }
    }
  }
}

// Joins the splits of one (row, head) in split order.
template <typename OT, int HD>
__global__ void __launch_bounds__(HD) k_attn_q8_join(AttnQ8 a) {
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.x, b = blockIdx.y, d = threadIdx.x;
  const int len = row_len(a, b);
  const int ns = (len + a.split_len - 1) / a.split_len;
  if (ns <= 1) return;
  float M = -CUDART_INF_F, L = 0.0f, A = 0.0f;
  const int64_t base = (int64_t)b * a.n_splits * a.H + h;
  for (int q = 0; q < ns; ++q) M = fmaxf(M, a.part_ml[2 * (base + (int64_t)q * a.H)]);
  for (int q = 0; q < ns; ++q) {
    const int64_t at = base + (int64_t)q * a.H;
    const float m = a.part_ml[2 * at];
    const float w = m == -CUDART_INF_F ? 0.0f : expf(m - M);
    L = fmaf(a.part_ml[2 * at + 1], w, L);
    A = fmaf(a.part_acc[at * HD + d], w, A);
  }
  st1(static_cast<OT*>(a.out) + b * a.out_stride + (int64_t)h * HD + d, L > 0.0f ? A / L : 0.0f);
}

template <typename QT, typename OT, int HD>
int launch_hd(const AttnQ8& a, cudaStream_t s) {
  launch_k(k_attn_q8<QT, OT, HD>, dim3(a.n_splits, a.kv.Hkv, a.n), kT, 0, s, a);
  if (a.n_splits == 1) return 1;
  launch_k(k_attn_q8_join<OT, HD>, dim3(a.H, a.n), HD, 0, s, a);
  return 2;
}

template <typename QT, typename OT>
int dispatch(const AttnQ8& a, cudaStream_t s) {
  switch (a.kv.hd) {
    case 64: return launch_hd<QT, OT, 64>(a, s);
    case 128: return launch_hd<QT, OT, 128>(a, s);
    case 256: return launch_hd<QT, OT, 256>(a, s);
    default: return 0;
  }
}

}  // namespace

// Enough splits for about eight blocks an SM, of at least 128 positions.
int attn_q8_split_len(int n, int Hkv, int max_len, int sms) {
  const int64_t pairs = std::max<int64_t>(1, (int64_t)n * Hkv);
  const int64_t want = std::max<int64_t>(1, 8 * (int64_t)sms / pairs);
  const int64_t len = (std::max(max_len, 1) + want - 1) / want;
  return (int)std::max<int64_t>(128, (len + 63) / 64 * 64);
}

int launch_attention_q8(const AttnQ8& a, int q_type, int out_type, cudaStream_t s) {
  if (a.n <= 0) return 0;
  if (q_type == X_BF16)
    return out_type == X_BF16 ? dispatch<__nv_bfloat16, __nv_bfloat16>(a, s)
                              : dispatch<__nv_bfloat16, float>(a, s);
  return out_type == X_BF16 ? dispatch<float, __nv_bfloat16>(a, s) : dispatch<float, float>(a, s);
}

}  // namespace fsk
