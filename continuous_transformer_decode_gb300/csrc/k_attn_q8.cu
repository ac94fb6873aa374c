// Attention of one new token a row over the 8-bit paged KV cache, split over
// the cache's length and joined.
//
//   o_h = sum_t p_t v_t,  p = softmax_t(scale * q_h . k_t),  t < length
//
// with k_t = ks_t * code, v_t = vs_t * code. The bytes are the codes, each wanted
// once; the work on a code (8 query heads at most) is far below the tensor
// cores' rate even of warp MMAs, so the kernel is bound by HBM if a code costs
// few instructions on its way. What that comes to:
//   * one block takes a split of one (row, KV head); each of its warps runs
//     through slices of 32 tokens with its own ring of stages filled by
//     cp.async, with no barrier in the loop;
//   * a byte becomes an f16 in one byte permute and half an addition: the byte
//     below 0x64 is 1024 + byte, less 1152 is the code, exact. (A bf16 would
//     take four instructions for two codes instead of two.)
//   * S = Q K^T and O += W V are m16n8k16 f16 MMAs. The order of the inner
//     index is free, so a thread's 16 bytes of a key row are its operands of four
//     k-steps, and 16 bytes of four value rows, interleaved by byte permutes,
//     those of sixteen n-tiles: no ldmatrix, no transpose. Rows 0..7 of A hold
//     the high f16 part of a head's q or weights and rows 8..15 what is left
//     (22 bits together), which costs nothing as a KV head has at most 8 heads;
//   * f16 is narrow, so q is brought to [2^13, 2^14) by a power of two per head,
//     and the weights w_t = exp2(s_t - R) vs_t are kept below 2^14 by a running
//     reference R, the maximum of s_t + log2(vs_t) less 13 (and not less than the
//     maximum of s less 126, for exp2's range), beside the softmax's own maximum
//     and sum. The scores are in log2 units.
// The warps, then the splits of a row (by a second kernel), are joined in order:
// a row's bits depend on its own inputs and split_len alone.

#include <math_constants.h>

#include <algorithm>

#include "attn_mma.cuh"
#include "kv_q8.cuh"

namespace fsk {
namespace {

using namespace attn;

constexpr int kWarps = 4;
constexpr int kT = 32 * kWarps;
constexpr int kG = 8;    // query heads per KV head at most
constexpr int kS = 32;   // tokens per slice
constexpr unsigned kAll = 0xffffffffu;
constexpr unsigned kNone = 0xffffffffu;  // no slot

template <int HD>
struct Lay {
  static constexpr int kStages = HD == 64 ? 4 : 3;  // slices in flight per warp, and one in use
  static constexpr int kK = kS * HD;                // bytes of a slice's key codes
  static constexpr int kStage = 2 * kK + 2 * kS * 4 + 16;  // codes, scales, mask of tokens
  static constexpr int kWarpBytes = kStages * kStage;
  static constexpr int kMerge = (int)sizeof(float) * (kG * HD + 2 * kG);  // a warp's (o, m, l)
  static constexpr int kBytes =
      kWarps * (kWarpBytes > kMerge ? kWarpBytes : kMerge) + (int)sizeof(float) * kG * (HD + 1);
};

// Byte offset of (row r < 32, 16-byte chunk c) in a slice's codes. The exclusive
// or spreads the 8 chunks that a quarter warp reads at once (two rows of keys,
// four of values) over all banks.
template <int HD>
__device__ __forceinline__ uint32_t at(int r, int c) {
  if constexpr (HD == 64) return (uint32_t)((r >> 1) * 128 + ((((r & 1) * 4 + c) ^ (r & 6)) << 4));
  return (uint32_t)(r * HD + ((c & ~7) << 4) + (((c & 7) ^ (r & 7)) << 4));
}

__device__ __forceinline__ float ld1(const float* p) { return *p; }
__device__ __forceinline__ float ld1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st1(float* p, float v) { *p = v; }
__device__ __forceinline__ void st1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Two codes (bytes lo and hi of w, chosen by the selector) as an f16 pair.
__device__ __forceinline__ uint32_t codes2(uint32_t w, uint32_t sel) {
  const uint32_t x = __byte_perm(w, 0x64646464u, sel);
  uint32_t y;
  asm("sub.f16x2 %0, %1, %2;" : "=r"(y) : "r"(x), "r"(0x64806480u));  // 1152, 1152
  return y;
}
__device__ __forceinline__ void split_f16(float x0, float x1, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 f = __half22float2(h);
  const __half2 l = __floats2half2_rn(x0 - f.x, x1 - f.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&l);
}
__device__ __forceinline__ void mma_f16(float d[4], const uint32_t a[4], uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Word w of a 16-byte vector (w a constant after unrolling).
__device__ __forceinline__ uint32_t word(const uint4& v, int w) {
  return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
}

__device__ __forceinline__ int row_len(const AttnQ8& a, int i) {
  return min(min(max(a.lens[i], 0), a.max_len), a.kv.max_pages * a.kv.page_size);
}

template <typename T, int HD>
__global__ void __launch_bounds__(kT, HD == 256 ? 1 : 2) k_attn_q8(AttnQ8 a) {
  using L = Lay<HD>;
  constexpr int kHalf = HD / 2;
  constexpr int kKs = HD / 16;         // k-steps of Q K^T
  constexpr int kNt = HD / 8;          // n-tiles of W V
  constexpr int kRowChunks = HD / 16;  // 16-byte chunks per row
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int H = a.H, G = H / a.kv.Hkv;
  const int len = row_len(a, b);
  const int start = s * a.split_len, end = min(len, start + a.split_len);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = lane >> 2, cq = lane & 3;
  T* orow = static_cast<T*>(a.out) + b * a.out_stride + (int64_t)g * G * HD;
  if (len == 0 && s == 0)
    for (int i = tid; i < G * HD; i += kT) st1(orow + i, 0.0f);
  if (start >= end) return;

  extern __shared__ __align__(128) uint8_t smem[];
  uint8_t* ring = smem + warp * L::kWarpBytes;
  float* qs = reinterpret_cast<float*>(smem + L::kBytes) - kG * (HD + 1);  // [kG][HD]
  float* qf = qs + kG * HD;                                                // [kG]

  // ---- the ring: slice i of this warp is tokens t0(i) .. t0(i) + 31
  const int n_slices = (end - start + kS - 1) / kS;
  const int mine = (n_slices - warp + kWarps - 1) / kWarps;
  const int row_lane = a.lanes[b];
  auto slot_of = [&](int i) -> unsigned {  // of token `lane` of slice i
    const int t = start + (i * kWarps + warp) * kS + lane;
    if (i >= mine || t >= end) return kNone;
    const int64_t x = q8::slot_of(a.kv, row_lane, t, g);
    return x < 0 ? kNone : (unsigned)x;
  };
  auto issue = [&](int i, unsigned slot) {
    uint8_t* st = ring + (i % L::kStages) * L::kStage;
    const uint32_t kb = smem_u32(st);
#pragma unroll
    for (int j = 0; j < kS * kRowChunks / 32; ++j) {
      const int x = lane + 32 * j, r = x / kRowChunks, c = x % kRowChunks;
      const unsigned sl = __shfl_sync(kAll, slot, r);
      if (sl != kNone) {
        const int64_t off = (int64_t)sl * HD + c * 16;
        cp_async16(kb + at<HD>(r, c), a.kv.k + off);
        cp_async16(kb + L::kK + at<HD>(r, c), a.kv.v + off);
      }
    }
    float* sc = reinterpret_cast<float*>(st + 2 * L::kK);  // [kS] ks, [kS] vs
    if (slot != kNone) {
      cp_async4(smem_u32(sc + lane), a.kv.ks + slot);
      cp_async4(smem_u32(sc + kS + lane), a.kv.vs + slot);
    } else {
      sc[lane] = sc[kS + lane] = 0.0f;
    }
    const unsigned mask = __ballot_sync(kAll, slot != kNone);
    if (lane == 0) *reinterpret_cast<unsigned*>(sc + 2 * kS) = mask;
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < L::kStages - 1; ++i) issue(i, slot_of(i));
  unsigned next_slot = slot_of(L::kStages - 1);

  // ---- q, rotated; warp w brings heads w, w + 4 to [2^13, 2^14)
  const T* qr = static_cast<const T*>(a.q) + b * a.q_stride + (int64_t)g * G * HD;
  for (int h = warp; h < kG; h += kWarps) {
    float x0[kHalf / 32], x1[kHalf / 32], mx = 0.0f;
#pragma unroll
    for (int j = 0; j < kHalf / 32; ++j) {
      const int i = lane + 32 * j;
      x0[j] = h < G ? ld1(qr + h * HD + i) : 0.0f;
      x1[j] = h < G ? ld1(qr + h * HD + i + kHalf) : 0.0f;
      if (a.rc) {
        const int64_t p = (int64_t)(len - 1) * kHalf + i;
        float y0, y1;
        rope_pair(x0[j], x1[j], a.rc[p], a.rs[p], y0, y1);
        x0[j] = y0;
        x1[j] = y1;
      }
      mx = fmaxf(mx, fmaxf(fabsf(x0[j]), fabsf(x1[j])));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, o));
    int e = 0;
    if (mx > 0.0f) frexpf(mx, &e);  // mx in [2^(e-1), 2^e)
    e = max(-110, min(e, 127)) - 14;
    const float up = ldexpf(1.0f, -e);
#pragma unroll
    for (int j = 0; j < kHalf / 32; ++j) {
      qs[h * HD + lane + 32 * j] = x0[j] * up;
      qs[h * HD + lane + 32 * j + kHalf] = x1[j] * up;
    }
    if (lane == 0) qf[h] = ldexpf(a.scale * 1.4426950408889634f, e);
  }
  __syncthreads();

  // A fragments: k-step 4 j + w of the thread holds elements 4 w .. 4 w + 3 of its
  // j-th chunk of 16
  auto chunk_of = [&](int j) {
    return HD == 64 ? cq : HD == 128 ? 2 * cq + j : 2 * cq + (j & 1) + 8 * (j >> 1);
  };
  uint32_t qa[kKs][4];
#pragma unroll
  for (int ks = 0; ks < kKs; ++ks) {
    const float* q = qs + gq * HD + chunk_of(ks / 4) * 16 + (ks % 4) * 4;
    split_f16(q[0], q[1], qa[ks][0], qa[ks][1]);
    split_f16(q[2], q[3], qa[ks][2], qa[ks][3]);
  }
  const float qfac = qf[gq];

  float m_run = -CUDART_INF_F, z_run = -CUDART_INF_F, ref = -CUDART_INF_F, l_run = 0.0f;
  float acc[kNt][4];
#pragma unroll
  for (int j = 0; j < kNt; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;

  for (int i = 0; i < mine; ++i) {
    // the stage that slice i - 1 was read from takes slice i + kStages - 1
    issue(i + L::kStages - 1, next_slot);
    next_slot = slot_of(i + L::kStages);
    cp_wait<L::kStages - 1>();
    __syncwarp();
    uint8_t* st = ring + (i % L::kStages) * L::kStage;
    const uint32_t kb = smem_u32(st), vb = kb + L::kK;
    const float* sc = reinterpret_cast<const float*>(st + 2 * L::kK);
    const unsigned mask = *reinterpret_cast<const unsigned*>(sc + 2 * kS);
    if (mask != 0) {
      // ---- scores of the slice, 4 n-tiles of 8 tokens
      float z[8], zs[8];
      float mx = -CUDART_INF_F, zx = -CUDART_INF_F;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < kKs / 4; ++j) {
          const uint4 kv = lds128(kb + at<HD>(8 * nt + gq, chunk_of(j)));
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const uint32_t x = word(kv, w);
            mma_f16(d, qa[4 * j + w], codes2(x, 0x4140u), codes2(x, 0x4342u));
          }
        }
        const float2 ks = *reinterpret_cast<const float2*>(sc + 8 * nt + 2 * cq);
        const float2 vs = *reinterpret_cast<const float2*>(sc + kS + 8 * nt + 2 * cq);
        const bool in0 = mask >> (8 * nt + 2 * cq) & 1, in1 = mask >> (8 * nt + 2 * cq + 1) & 1;
        z[2 * nt] = in0 ? (d[0] + d[2]) * (ks.x * qfac) : -CUDART_INF_F;
        z[2 * nt + 1] = in1 ? (d[1] + d[3]) * (ks.y * qfac) : -CUDART_INF_F;
        zs[2 * nt] = vs.x;
        zs[2 * nt + 1] = vs.y;
        mx = fmaxf(mx, fmaxf(z[2 * nt], z[2 * nt + 1]));
        zx = fmaxf(zx, fmaxf(z[2 * nt] + lg2(vs.x), z[2 * nt + 1] + lg2(vs.y)));
      }
      // ---- running maximum and reference of the head (its four threads)
      mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 1));
      zx = fmaxf(zx, __shfl_xor_sync(kAll, zx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 2));
      zx = fmaxf(zx, __shfl_xor_sync(kAll, zx, 2));
      if (__any_sync(kAll, mx > m_run || zx > z_run)) {
        const float m_new = fmaxf(m_run, mx);
        z_run = fmaxf(z_run, zx);
        const float r_new = fmaxf(z_run - 13.0f, m_new - 126.0f);
        l_run *= m_run == -CUDART_INF_F ? 0.0f : ex2(m_run - m_new);
        const float f = ref == -CUDART_INF_F ? 0.0f : ex2(ref - r_new);
        m_run = m_new;
        ref = r_new;
#pragma unroll
        for (int j = 0; j < kNt; ++j) {
          acc[j][0] *= f;
          acc[j][1] *= f;
          acc[j][2] *= f;
          acc[j][3] *= f;
        }
      }
      // ---- weights, and O += W V in two k-steps of 16 tokens
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          l_run += ex2(z[4 * kk + e] - m_run);
          w[e] = ex2(z[4 * kk + e] - ref) * zs[4 * kk + e];
        }
        uint32_t wa[4];
        split_f16(w[0], w[1], wa[0], wa[1]);
        split_f16(w[2], w[3], wa[2], wa[3]);
        // rows r0, r0 + 1, r0 + 8, r0 + 9; the thread's HD / 8 columns
        const int r0 = 16 * kk + 2 * cq;
        if constexpr (HD == 64) {
          const int c = gq >> 1, o = (gq & 1) * 8;
          const uint2 v0 = lds64(vb + at<HD>(r0, c) + o), v1 = lds64(vb + at<HD>(r0 + 1, c) + o);
          const uint2 v2 = lds64(vb + at<HD>(r0 + 8, c) + o), v3 = lds64(vb + at<HD>(r0 + 9, c) + o);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t a0 = x ? v0.y : v0.x, a1 = x ? v1.y : v1.x;
            const uint32_t a2 = x ? v2.y : v2.x, a3 = x ? v3.y : v3.x;
            const uint32_t p0 = __byte_perm(a0, a1, 0x5140), p1 = __byte_perm(a0, a1, 0x7362);
            const uint32_t p2 = __byte_perm(a2, a3, 0x5140), p3 = __byte_perm(a2, a3, 0x7362);
            mma_f16(acc[4 * x], wa, codes2(p0, 0x4140u), codes2(p2, 0x4140u));
            mma_f16(acc[4 * x + 1], wa, codes2(p0, 0x4342u), codes2(p2, 0x4342u));
            mma_f16(acc[4 * x + 2], wa, codes2(p1, 0x4140u), codes2(p3, 0x4140u));
            mma_f16(acc[4 * x + 3], wa, codes2(p1, 0x4342u), codes2(p3, 0x4342u));
          }
        } else {
#pragma unroll
          for (int jj = 0; jj < HD / 128; ++jj) {
            const int c = gq + 8 * jj;
            const uint4 v0 = lds128(vb + at<HD>(r0, c)), v1 = lds128(vb + at<HD>(r0 + 1, c));
            const uint4 v2 = lds128(vb + at<HD>(r0 + 8, c)), v3 = lds128(vb + at<HD>(r0 + 9, c));
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t a0 = word(v0, x), a1 = word(v1, x), a2 = word(v2, x), a3 = word(v3, x);
              const uint32_t p0 = __byte_perm(a0, a1, 0x5140), p1 = __byte_perm(a0, a1, 0x7362);
              const uint32_t p2 = __byte_perm(a2, a3, 0x5140), p3 = __byte_perm(a2, a3, 0x7362);
              float(*o)[4] = acc + 16 * jj + 4 * x;
              mma_f16(o[0], wa, codes2(p0, 0x4140u), codes2(p2, 0x4140u));
              mma_f16(o[1], wa, codes2(p0, 0x4342u), codes2(p2, 0x4342u));
              mma_f16(o[2], wa, codes2(p1, 0x4140u), codes2(p3, 0x4140u));
              mma_f16(o[3], wa, codes2(p1, 0x4342u), codes2(p3, 0x4342u));
            }
          }
        }
      }
    }
    __syncwarp();  // every lane has read the stage that the next issue fills
  }
  l_run += __shfl_xor_sync(kAll, l_run, 1);
  l_run += __shfl_xor_sync(kAll, l_run, 2);

  // ---- join the warps in order, through the idle rings
  __syncthreads();
  float* wo = reinterpret_cast<float*>(smem);  // [kWarps][kG][HD], then m and l [kWarps][kG]
  float* wm = wo + kWarps * kG * HD;
  float* wl = wm + kWarps * kG;
  const float back = m_run == -CUDART_INF_F ? 0.0f : ex2(ref - m_run);
  if (gq < G) {
    float* o = wo + (warp * kG + gq) * HD;
#pragma unroll
    for (int j = 0; j < kNt; ++j) {
      // n-tile j's columns 2 cq, 2 cq + 1 are chunks of those thread rows, byte j
      const int d0 = HD == 64 ? 2 * cq * 8 + j : (2 * cq + 8 * (j / 16)) * 16 + j % 16;
      const int d1 = d0 + (HD == 64 ? 8 : 16);
      o[d0] = (acc[j][0] + acc[j][2]) * back;
      o[d1] = (acc[j][1] + acc[j][3]) * back;
    }
    if (cq == 0) {
      wm[warp * kG + gq] = m_run;
      wl[warp * kG + gq] = l_run;
    }
  }
  __syncthreads();
  const int64_t base = ((int64_t)b * a.n_splits + s) * H + g * G;
  for (int i = tid; i < G * HD; i += kT) {
    const int h = i / HD, d = i % HD;
    float M = -CUDART_INF_F, Lsum = 0.0f, A = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, wm[w * kG + h]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float m = wm[w * kG + h], f = m == -CUDART_INF_F ? 0.0f : ex2(m - M);
      Lsum = fmaf(wl[w * kG + h], f, Lsum);
      A = fmaf(wo[(w * kG + h) * HD + d], f, A);
    }
    if (len <= a.split_len) {
      st1(orow + i, Lsum > 0.0f ? A / Lsum : 0.0f);
    } else {
      a.part_acc[base * HD + i] = A;
      if (d == 0) {
        a.part_ml[2 * (base + h)] = M;
        a.part_ml[2 * (base + h) + 1] = Lsum;
      }
    }
  }
}

// Joins the splits of one (row, head) in split order.
template <typename T, int HD>
__global__ void __launch_bounds__(HD) k_attn_q8_join(AttnQ8 a) {
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.x, b = blockIdx.y, d = threadIdx.x;
  const int len = row_len(a, b);
  const int ns = (len + a.split_len - 1) / a.split_len;
  if (ns <= 1) return;
  float M = -CUDART_INF_F, Lsum = 0.0f, A = 0.0f;
  const int64_t base = (int64_t)b * a.n_splits * a.H + h;
  for (int q = 0; q < ns; ++q) M = fmaxf(M, a.part_ml[2 * (base + (int64_t)q * a.H)]);
  for (int q = 0; q < ns; ++q) {
    const int64_t x = base + (int64_t)q * a.H;
    const float m = a.part_ml[2 * x], f = m == -CUDART_INF_F ? 0.0f : ex2(m - M);
    Lsum = fmaf(a.part_ml[2 * x + 1], f, Lsum);
    A = fmaf(a.part_acc[x * HD + d], f, A);
  }
  st1(static_cast<T*>(a.out) + b * a.out_stride + (int64_t)h * HD + d,
      Lsum > 0.0f ? A / Lsum : 0.0f);
}

template <typename T, int HD>
int launch_hd(const AttnQ8& a, cudaStream_t s) {
  // per device, so set on every call (a host-side store, well below a launch)
  cudaFuncSetAttribute(k_attn_q8<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       Lay<HD>::kBytes);
  launch_k(k_attn_q8<T, HD>, dim3(a.n_splits, a.kv.Hkv, a.n), kT, Lay<HD>::kBytes, s, a);
  if (a.n_splits == 1) return 1;
  launch_k(k_attn_q8_join<T, HD>, dim3(a.H, a.n), HD, 0, s, a);
  return 2;
}

template <typename T>
int dispatch(const AttnQ8& a, cudaStream_t s) {
  switch (a.kv.hd) {
    case 64: return launch_hd<T, 64>(a, s);
    case 128: return launch_hd<T, 128>(a, s);
    case 256: return launch_hd<T, 256>(a, s);
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

int launch_attention_q8(const AttnQ8& a, int x_type, cudaStream_t s) {
  if (a.n <= 0) return 0;
  return x_type == X_BF16 ? dispatch<__nv_bfloat16>(a, s) : dispatch<float>(a, s);
}

}  // namespace fsk
