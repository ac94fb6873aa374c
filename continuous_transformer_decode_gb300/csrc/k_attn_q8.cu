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
//     through slices of 32 tokens (16 at head_dim 256) with its own ring of
//     stages filled by cp.async, with no barrier in the loop; the page of a
//     slice is looked up one slice before its copies are issued;
//   * a byte becomes an f16 in one byte permute and half an addition: the byte
//     below 0x64 is 1024 + byte, less 1152 is the code, exact. (A bf16 would
//     take four instructions for two codes instead of two.)
//   * S = Q K^T and O^T += V^T W are m16n8k16 f16 MMAs. The order of the inner
//     index is free, so a thread's 16 bytes of a key row are its operands of four
//     k-steps, and 16 bytes of four value rows, interleaved by byte permutes,
//     those of eight m-tiles: no ldmatrix, no transpose. q and the weights are two
//     f16 parts (22 bits): of q in rows 0..7 and 8..15 of A, which costs nothing
//     as a KV head has at most 8 heads; of the weights in two MMAs into one
//     accumulator, half the registers of W V with its two parts in rows;
//   * f16 is narrow, so q is brought to [2^13, 2^14) by a power of two per head,
//     and the weights w_t = exp2(s_t - R) vs_t are kept in f16's range by a
//     reference R per head: the maximum of s_t + log2(vs_t) less 13 when it was
//     set (and not less than the maximum of s less 110, for exp2's range), set
//     anew only when a weight would pass 2^15.9. The softmax's sum has a reference of its
//     own, m. So most slices look at their scores with one vote, and neither
//     shuffle a maximum nor rescale the accumulators. Scores are in log2 units;
//     the largest weight is at least 2^13 in f16 (values below 2^-97 apart), so
//     each is held to 2^-22 of itself or 2^-38 of the largest.
// The warps, then the splits of a row (by a second kernel), are joined in order:
// a row's bits depend on its own inputs and split_len alone.

#include <math_constants.h>

#include <algorithm>

#include "attn_mma.cuh"
#include "kv_q8.cuh"

namespace fsk {
FS_TRACE_TU(attn_q8)
namespace {

using namespace attn;

constexpr int kG = 8;    // query heads per KV head at most
constexpr unsigned kAll = 0xffffffffu;

// Warps of a block, blocks an SM, tokens of a slice, and stages of a warp's ring
// (one in use, the others in flight).
template <int HD>
struct Shape;
template <>
struct Shape<64> {
  static constexpr int kWarps = 4, kBlocks = 5, kS = 32, kStages = 2;
};
template <>
struct Shape<128> {
  static constexpr int kWarps = 4, kBlocks = 3, kS = 32, kStages = 2;
};
template <>
struct Shape<256> {
  static constexpr int kWarps = 8, kBlocks = 1, kS = 16, kStages = 3;
};

template <int HD>
struct Lay : Shape<HD> {
  using Shape<HD>::kWarps;
  using Shape<HD>::kS;
  using Shape<HD>::kStages;
  static constexpr int kT = 32 * kWarps;
  static constexpr int kK = kS * HD;                 // bytes of a slice's key codes
  static constexpr int kStage = 2 * kK + 2 * kS * 4 + 16;  // codes, scales, mask of tokens
  static constexpr int kWarpBytes = kStages * kStage;
  static constexpr int kMerge = (int)sizeof(float) * (kG * HD + 2 * kG);  // a warp's (o, m, l)
  static constexpr int kQa = HD / 16 * 32 * 16;  // q's A fragments, 16 bytes a lane and k-step
  static constexpr int kBytes =
      kWarps * (kWarpBytes > kMerge ? kWarpBytes : kMerge) + kQa + (int)sizeof(float) * kG;
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
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds128(const uint8_t* p) {
  return *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ uint2 lds64(const uint8_t* p) {
  return *reinterpret_cast<const uint2*>(p);
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
// NaN if one of them is: a head whose q is not a number gives no number.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
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
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two m-tiles of V^T W: a0 .. a3 are the same four columns (bytes) of tokens 2 cq,
// 2 cq + 1, 2 cq + 8, 2 cq + 9; interleaved by twos they are the A operands,
// columns 0 and 1 rows gq and gq + 8 of the first tile, 2 and 3 of the second.
// w: the head's weights of these tokens (hi 0 1, lo 0 1, hi 2 3, lo 2 3).
__device__ __forceinline__ void value_tiles(float (*o)[4], const uint32_t w[4], uint32_t a0,
                                            uint32_t a1, uint32_t a2, uint32_t a3) {
  const uint32_t p0 = __byte_perm(a0, a1, 0x5140), p1 = __byte_perm(a0, a1, 0x7362);
  const uint32_t p2 = __byte_perm(a2, a3, 0x5140), p3 = __byte_perm(a2, a3, 0x7362);
  const uint32_t x[4] = {codes2(p0, 0x4140u), codes2(p0, 0x4342u), codes2(p2, 0x4140u),
                         codes2(p2, 0x4342u)};
  const uint32_t y[4] = {codes2(p1, 0x4140u), codes2(p1, 0x4342u), codes2(p3, 0x4140u),
                         codes2(p3, 0x4342u)};
  mma_f16(o[0], x, w[0], w[2]);
  mma_f16(o[1], y, w[0], w[2]);
  mma_f16(o[0], x, w[1], w[3]);
  mma_f16(o[1], y, w[1], w[3]);
}
// Word w of a 16-byte vector (w a constant after unrolling).
__device__ __forceinline__ uint32_t word(const uint4& v, int w) {
  return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
}

__device__ __forceinline__ int row_len(const AttnQ8& a, int i) {
  return min(max(a.lens[i], 0), a.max_len - a.len_add) + a.len_add;
}

// The row whose length is the rank-th largest (ties: the lower row first), found by
// every block for itself: blocks start in about the order of their indexes, so the
// long rows start first and the SMs finish together: 128 lanes of 128 to 4096 tokens
// take 94 us instead of 108, 192 lanes 142 instead of 144. Comparing all rows costs a
// block one to three microseconds and more with more rows (256 lanes would take 190
// instead of 185), so it is for at most 192 rows, in launches of at least two blocks a
// place whose blocks may be long (256 lanes of up to 512 tokens would take 19 us instead
// of 13). max_len stands for the lengths, which the host does not know: 128 rows of 200
// tokens under a max_len of 4096 pay for nothing, 27 us instead of 23.
constexpr int kRankRows = 192;  // most rows that this is done for
template <int kT>
__device__ __forceinline__ int row_of_rank(const AttnQ8& a, int rank, uint8_t* smem) {
  // keys that differ: the length (up to 2^22), then the row
  int* key = reinterpret_cast<int*>(smem);
  const int4* key4 = reinterpret_cast<const int4*>(smem);
  __shared__ int row;
  for (int i = threadIdx.x; i < (a.n + 3) / 4 * 4; i += kT)
    key[i] = i < a.n ? min(max(a.lens[i], 0), 1 << 22) * kRankRows + (kRankRows - 1 - i) : -1;
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += kT) {
    const int mine = key[i];
    int ahead[4] = {0, 0, 0, 0};
#pragma unroll 4
    for (int j = 0; j < (a.n + 3) / 4; ++j) {
      const int4 v = key4[j];
      ahead[0] += v.x > mine;
      ahead[1] += v.y > mine;
      ahead[2] += v.z > mine;
      ahead[3] += v.w > mine;
    }
    if (ahead[0] + ahead[1] + ahead[2] + ahead[3] == rank) row = i;
  }
  __syncthreads();
  return row;
}

template <typename QT, typename OT, int HD>
__device__ __forceinline__ void attn_q8_body(const AttnQ8& a) {
  using L = Lay<HD>;
  constexpr int kWarps = L::kWarps, kT = L::kT, kS = L::kS;
  constexpr int kHalf = HD / 2;
  constexpr int kKs = HD / 16;         // k-steps of Q K^T
  constexpr int kMt = HD / 16;         // m-tiles of V^T W
  constexpr int kRowChunks = HD / 16;  // 16-byte chunks per row
  const int g = blockIdx.x, s = blockIdx.z;
  extern __shared__ __align__(128) uint8_t smem[];
  const int b = a.by_len ? row_of_rank<kT>(a, blockIdx.y, smem) : blockIdx.y;
  const int H = a.H, G = H / a.kv.Hkv;
  // a block's loads depend on one another three deep: (length, lane, q), then (pages,
  // rotation), then codes; each level is asked for together
  const int row_lane = a.lanes[b];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const QT* qr = static_cast<const QT*>(a.q) + b * a.q_stride + (int64_t)g * G * HD;
  constexpr int kHeads = (kG + kWarps - 1) / kWarps, kP = kHalf / 32;
  float x0[kHeads][kP], x1[kHeads][kP];  // warp w takes heads w, w + kWarps, ..
#pragma unroll
  for (int u = 0; u < kHeads; ++u)
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      const int h = warp + u * kWarps, i = lane + 32 * j;
      x0[u][j] = h < G ? ld1(qr + h * HD + i) : 0.0f;
      x1[u][j] = h < G ? ld1(qr + h * HD + i + kHalf) : 0.0f;
    }
  const int len = row_len(a, b);
  const int start = s * a.split_len, end = min(len, start + a.split_len);
  const int gq = lane >> 2, cq = lane & 3;
  OT* orow = static_cast<OT*>(a.out) + b * a.out_stride + (int64_t)g * G * HD;
  if (len == 0 && s == 0)
    for (int i = tid; i < G * HD; i += kT) st_out(orow + i, 0.0f, a.out_lo);
  if (start >= end) return;

  uint8_t* ring = smem + warp * L::kWarpBytes;
  uint8_t* qa = smem + L::kBytes - L::kQa - (int)sizeof(float) * kG;  // [kKs][32] uint4
  float* qf = reinterpret_cast<float*>(qa + L::kQa);                  // [kG]

  // ---- the ring: slice i of this warp is tokens t0(i) .. t0(i) + kS - 1; lane l
  // follows token t0(i) + l, its page in the lane's table and its slot in the page
  const int n_slices = (end - start + kS - 1) / kS;
  const int mine = (n_slices - warp + kWarps - 1) / kWarps;
  const int ps = a.kv.page_size;
  const bool no_lane = (unsigned)row_lane >= (unsigned)a.kv.n_lanes;
  const int32_t* pages = a.kv.page_table + (no_lane ? 0 : (int64_t)row_lane * a.kv.max_pages);
  constexpr int kStep = kWarps * kS;
  const int step_page = (int)a.kv.by_page.div(kStep), step_slot = kStep - step_page * ps;
  int t_next = start + warp * kS + lane;
  int p_next = (int)a.kv.by_page.div(t_next), s_next = t_next - p_next * ps;
  // (page as the table has it, slot) of this lane's token of the next slice; -1: no token
  auto look_up = [&](int& page, int& slot) {
    page = lane < kS && t_next < end && !no_lane ? pages[p_next] : -1;
    slot = s_next;
    t_next += kStep;
    p_next += step_page;
    s_next += step_slot;
    if (s_next >= ps) {
      s_next -= ps;
      ++p_next;
    }
  };
  auto issue = [&](uint8_t* st, int page, int in_page) {
    const uint32_t kb = smem_u32(st);
    const bool in = (unsigned)page < (unsigned)a.kv.n_pages;
    const unsigned slot = ((unsigned)page * a.kv.Hkv + g) * ps + in_page;
    const unsigned mask = __ballot_sync(kAll, in);
#pragma unroll
    for (int j = 0; j < kS * kRowChunks / 32; ++j) {
      const int x = lane + 32 * j, r = x / kRowChunks, c = x % kRowChunks;
      const unsigned sl = __shfl_sync(kAll, slot, r);
      if (mask >> r & 1) {
        const int64_t off = (int64_t)sl * HD + c * 16;
        cp_async16(kb + at<HD>(r, c), a.kv.k + off);
        cp_async16(kb + L::kK + at<HD>(r, c), a.kv.v + off);
      }
    }
    float* sc = reinterpret_cast<float*>(st + 2 * L::kK);  // [kS] ks, [kS] vs
    if (in) {
      cp_async4(smem_u32(sc + lane), a.kv.ks + slot);
      cp_async4(smem_u32(sc + kS + lane), a.kv.vs + slot);
    } else if (lane < kS) {
      sc[lane] = sc[kS + lane] = 0.0f;
    }
    if (lane == 0) *reinterpret_cast<unsigned*>(sc + 2 * kS) = mask;
    cp_commit();
  };
  int page[L::kStages], slot[L::kStages];
#pragma unroll
  for (int i = 0; i < L::kStages; ++i) look_up(page[i], slot[i]);

  float rc[kP], rs[kP];
#pragma unroll
  for (int j = 0; j < kP; ++j) {
    const int64_t p = (int64_t)(len - 1) * kHalf + lane + 32 * j;
    rc[j] = a.rc ? a.rc[p] : 1.0f;
    rs[j] = a.rc ? a.rs[p] : 0.0f;
  }
#pragma unroll
  for (int i = 0; i < L::kStages - 1; ++i) issue(ring + i * L::kStage, page[i], slot[i]);
  int next_page = page[L::kStages - 1], next_slot = slot[L::kStages - 1];

  // ---- q, rotated, into A fragments
  // element d of head h in the A fragments: chunk d / 16 is the j-th chunk of thread
  // column cq, and word w of it (elements 4 w .. 4 w + 3) k-step 4 j + w; the
  // lane's 16 bytes are (hi 0 1, lo 0 1, hi 2 3, lo 2 3)
  auto put_q = [&](int h, int d, float x) {
    const int chunk = d / 16, w = d % 16 / 4, e = d % 4;
    const int c = HD == 64 ? chunk : (chunk % 8) / 2;
    const int j = HD == 64 ? 0 : chunk % 2 + chunk / 8 * 2;
    const __half hi = __float2half_rn(x);
    __half* f = reinterpret_cast<__half*>(qa + ((4 * j + w) * 32 + h * 4 + c) * 16) + (e & 1) + (e & 2) * 2;
    f[0] = hi;
    f[2] = __float2half_rn(x - __half2float(hi));
  };
#pragma unroll
  for (int u = 0; u < kHeads; ++u) {
    const int h = warp + u * kWarps;
    if (h >= kG) break;
    float mx = 0.0f;
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      float y0 = x0[u][j], y1 = x1[u][j];
      if (a.rc) rope_pair(x0[u][j], x1[u][j], rc[j], rs[j], y0, y1);
      x0[u][j] = y0;
      x1[u][j] = y1;
      mx = fmaxf(mx, fmaxf(fabsf(y0), fabsf(y1)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, o));
    // mx in [2^(e + 13), 2^(e + 14)), by its exponent; -124 <= e <= 114
    const int e = max((int)(__float_as_uint(mx) >> 23) - 127, -111) - 13;
    const float up = __uint_as_float((unsigned)(127 - e) << 23);  // 2^-e
#pragma unroll
    for (int j = 0; j < kP; ++j) {
      put_q(h, lane + 32 * j, x0[u][j] * up);
      put_q(h, lane + 32 * j + kHalf, x1[u][j] * up);
    }
    if (lane == 0)
      qf[h] = a.scale * 1.4426950408889634f * __uint_as_float((unsigned)(127 + e) << 23);
  }
  __syncthreads();

  auto chunk_of = [&](int j) {
    return HD == 64 ? cq : HD == 128 ? 2 * cq + j : 2 * cq + (j & 1) + 8 * (j >> 1);
  };
  const float qfac = qf[gq];
  constexpr float kTop = 15.9f;  // a weight may reach 2^kTop before R is set anew
  float m_ref = -CUDART_INF_F, ref = -CUDART_INF_F, l_run = 0.0f;
  float acc[kMt][4];  // [tile][(column 0, column 1) x (head 2 cq, head 2 cq + 1)]
#pragma unroll
  for (int j = 0; j < kMt; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.0f;

  int use = 0, fill = L::kStages - 1;  // stages: of this slice, and of the next to issue
  for (int i = 0; i < mine; ++i) {
    // the stage that the last slice was read from takes slice i + kStages - 1
    issue(ring + fill * L::kStage, next_page, next_slot);
    look_up(next_page, next_slot);
    cp_wait<L::kStages - 1>();
    __syncwarp();
    const uint8_t* kb = ring + use * L::kStage;
    const uint8_t* vb = kb + L::kK;
    const float* sc = reinterpret_cast<const float*>(kb + 2 * L::kK);
    const unsigned mask = *reinterpret_cast<const unsigned*>(sc + 2 * kS);
    fill = use;
    use = use + 1 == L::kStages ? 0 : use + 1;
    if (mask != 0) {
      // ---- scores of the slice, n-tiles of 8 tokens
      float z[kS / 4], zs[kS / 4];
      float mx = -CUDART_INF_F, zx = -CUDART_INF_F;
      float d[kS / 8][4];
#pragma unroll
      for (int nt = 0; nt < kS / 8; ++nt) d[nt][0] = d[nt][1] = d[nt][2] = d[nt][3] = 0.0f;
#pragma unroll
      for (int j = 0; j < kKs / 4; ++j) {
        uint4 kv[kS / 8];
#pragma unroll
        for (int nt = 0; nt < kS / 8; ++nt) kv[nt] = lds128(kb + at<HD>(8 * nt + gq, chunk_of(j)));
#pragma unroll
        for (int w = 0; w < 4; ++w) {  // the n-tiles in turn: independent chains of MMAs
          const uint4 q4 = lds128(qa + ((4 * j + w) * 32 + lane) * 16);
          const uint32_t fr[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
          for (int nt = 0; nt < kS / 8; ++nt) {
            const uint32_t x = word(kv[nt], w);
            mma_f16(d[nt], fr, codes2(x, 0x4140u), codes2(x, 0x4342u));
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < kS / 8; ++nt) {
        const float2 ks = *reinterpret_cast<const float2*>(sc + 8 * nt + 2 * cq);
        const float2 vs = *reinterpret_cast<const float2*>(sc + kS + 8 * nt + 2 * cq);
        z[2 * nt] = (d[nt][0] + d[nt][2]) * (ks.x * qfac);
        z[2 * nt + 1] = (d[nt][1] + d[nt][3]) * (ks.y * qfac);
        zs[2 * nt] = vs.x;
        zs[2 * nt + 1] = vs.y;
      }
      if (mask != (kS == 32 ? kAll : (1u << (kS & 31)) - 1)) {  // a slice with absent tokens
#pragma unroll
        for (int e = 0; e < kS / 4; ++e)
          if (!(mask >> (8 * (e / 2) + 2 * cq + e % 2) & 1)) z[e] = -CUDART_INF_F;
      }
#pragma unroll
      for (int e = 0; e < kS / 4; ++e) {
        mx = max_nan(mx, z[e]);
        zx = fmaxf(zx, z[e] + lg2(zs[e]));
      }
      if (__any_sync(kAll, !(mx <= m_ref + kTop) || zx > ref + kTop)) {
        // the head's maxima (its four threads), and new references
        mx = max_nan(mx, __shfl_xor_sync(kAll, mx, 1));
        zx = fmaxf(zx, __shfl_xor_sync(kAll, zx, 1));
        mx = max_nan(mx, __shfl_xor_sync(kAll, mx, 2));
        zx = fmaxf(zx, __shfl_xor_sync(kAll, zx, 2));
        const float m_new = max_nan(m_ref, mx);
        const float r_new = fmaxf(ref, fmaxf(zx - 13.0f, m_new - 110.0f));
        l_run *= m_ref == -CUDART_INF_F ? 0.0f : ex2(m_ref - m_new);
        const float f = ref == -CUDART_INF_F ? 0.0f : ex2(ref - r_new);
        m_ref = m_new;
        ref = r_new;
        const float f0 = __shfl_sync(kAll, f, 8 * cq), f1 = __shfl_sync(kAll, f, 8 * cq + 4);
#pragma unroll
        for (int j = 0; j < kMt; ++j) {
          acc[j][0] *= f0;
          acc[j][1] *= f1;
          acc[j][2] *= f0;
          acc[j][3] *= f1;
        }
      }
      // ---- weights, and O^T += V^T W in k-steps of 16 tokens
#pragma unroll
      for (int kk = 0; kk < kS / 16; ++kk) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          l_run += ex2(z[4 * kk + e] - m_ref);
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
          for (int x = 0; x < 2; ++x)
            value_tiles(acc + 2 * x, wa, x ? v0.y : v0.x, x ? v1.y : v1.x, x ? v2.y : v2.x,
                        x ? v3.y : v3.x);
        } else {
#pragma unroll
          for (int jj = 0; jj < HD / 128; ++jj) {
            const int c = gq + 8 * jj;
            const uint4 v0 = lds128(vb + at<HD>(r0, c)), v1 = lds128(vb + at<HD>(r0 + 1, c));
            const uint4 v2 = lds128(vb + at<HD>(r0 + 8, c)), v3 = lds128(vb + at<HD>(r0 + 9, c));
#pragma unroll
            for (int x = 0; x < 4; ++x)
              value_tiles(acc + 8 * jj + 2 * x, wa, word(v0, x), word(v1, x), word(v2, x),
                          word(v3, x));
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
  const float back = m_ref == -CUDART_INF_F ? 0.0f : ex2(ref - m_ref);
  const float back0 = __shfl_sync(kAll, back, 8 * cq), back1 = __shfl_sync(kAll, back, 8 * cq + 4);
  float* o0 = wo + (warp * kG + 2 * cq) * HD;  // heads 2 cq and 2 cq + 1
#pragma unroll
  for (int j = 0; j < kMt; ++j) {  // tile j holds columns 2 j, 2 j + 1 of the thread's chunks
    const int col = HD == 64 ? 8 * gq + 2 * j : (gq + 8 * (j / 8)) * 16 + 2 * (j % 8);
    *reinterpret_cast<float2*>(o0 + col) = make_float2(acc[j][0] * back0, acc[j][2] * back0);
    *reinterpret_cast<float2*>(o0 + HD + col) = make_float2(acc[j][1] * back1, acc[j][3] * back1);
  }
  if (cq == 0) {
    wm[warp * kG + gq] = m_ref;
    wl[warp * kG + gq] = l_run;
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
      st_out(orow + i, Lsum == 0.0f ? 0.0f : A / Lsum, a.out_lo);
    } else {
      a.part_acc[base * HD + i] = A;
      if (d == 0) {
        a.part_ml[2 * (base + h)] = M;
        a.part_ml[2 * (base + h) + 1] = Lsum;
      }
    }
  }
}

template <typename QT, typename OT, int HD, bool kTrace>
__global__ void __launch_bounds__(Lay<HD>::kT, Lay<HD>::kBlocks) k_attn_q8(AttnQ8 a) {
  __shared__ unsigned long long s_tr[kTrace ? 4 : 1];
  if constexpr (kTrace) TraceSmem::begin(s_tr, g_trace);
  pdl_wait();
  if constexpr (kTrace) TraceSmem::ready(s_tr);
  pdl_trigger();
  attn_q8_body<QT, OT, HD>(a);
  if constexpr (kTrace) TraceSmem::end(s_tr, TR_ATTN_Q8);
}

// Joins the splits of one (row, head): the weights of the splits first, then
// HD / 4 columns of threads by kJ, column x taking splits x, x + kJ, .. in
// order, and the kJ sums in order.
constexpr int kJ = 8;
template <typename OT, int HD, bool kTrace>
__global__ void __launch_bounds__(HD / 4 * kJ) k_attn_q8_join(AttnQ8 a) {
  TraceScope tr(kTrace ? g_trace : nullptr, TR_ATTN_Q8_JOIN);
  constexpr int kT = HD / 4 * kJ;
  __shared__ float4 part[kJ][HD / 4];
  __shared__ float red[2][kT / 32];
  extern __shared__ float w[];  // [n_splits]
  pdl_wait();
  tr.ready();
  pdl_trigger();
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  const int len = row_len(a, b);
  const int ns = (len + a.split_len - 1) / a.split_len;
  if (ns <= 1) return;
  const int64_t base = (int64_t)b * a.n_splits * a.H + h;
  float M = -CUDART_INF_F;
  for (int q = tid; q < ns; q += kT) {
    w[q] = a.part_ml[2 * (base + (int64_t)q * a.H)];
    M = fmaxf(M, w[q]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
  if (tid % 32 == 0) red[0][tid / 32] = M;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kT / 32; ++i) M = fmaxf(M, red[0][i]);
  float Lsum = 0.0f;
  for (int q = tid; q < ns; q += kT) {
    const float f = w[q] == -CUDART_INF_F ? 0.0f : ex2(w[q] - M);
    w[q] = f;
    Lsum = fmaf(a.part_ml[2 * (base + (int64_t)q * a.H) + 1], f, Lsum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) Lsum += __shfl_xor_sync(kAll, Lsum, o);
  if (tid % 32 == 0) red[1][tid / 32] = Lsum;
  __syncthreads();
  const int col = tid % (HD / 4), x = tid / (HD / 4);
  float4 A = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float4* src = reinterpret_cast<const float4*>(a.part_acc) + base * (HD / 4) + col;
#pragma unroll 4
  for (int q = x; q < ns; q += kJ) {
    const float4 v = src[(int64_t)q * a.H * (HD / 4)];
    A.x = fmaf(v.x, w[q], A.x);
    A.y = fmaf(v.y, w[q], A.y);
    A.z = fmaf(v.z, w[q], A.z);
    A.w = fmaf(v.w, w[q], A.w);
  }
  part[x][col] = A;
  __syncthreads();
  if (tid >= HD) return;
  Lsum = 0.0f;
#pragma unroll
  for (int i = 0; i < kT / 32; ++i) Lsum += red[1][i];
  float o = 0.0f;
#pragma unroll
  for (int i = 0; i < kJ; ++i) o += reinterpret_cast<const float*>(part[i])[tid];
  st_out(static_cast<OT*>(a.out) + b * a.out_stride + (int64_t)h * HD + tid,
         Lsum == 0.0f ? 0.0f : o / Lsum, a.out_lo);
}

template <typename QT, typename OT, int HD, bool kTrace>
Launched launch_hd(const AttnQ8& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  auto kern = k_attn_q8<QT, OT, HD, kTrace>;
  Launched l;
  l.error = allow_smem(kern, Lay<HD>::kBytes, done);
  if (l.error == cudaSuccess &&
      l.add(launch_k(kern, dim3(a.kv.Hkv, a.n, a.n_splits), Lay<HD>::kT, Lay<HD>::kBytes, s, a)) &&
      a.n_splits > 1)
    l.add(launch_k(k_attn_q8_join<OT, HD, kTrace>, dim3(a.H, a.n), HD / 4 * kJ, a.n_splits * sizeof(float),
                   s, a));
  return l;
}

template <typename QT, typename OT, bool kTrace>
Launched dispatch(const AttnQ8& a, cudaStream_t s) {
  switch (a.kv.hd) {
    case 64: return launch_hd<QT, OT, 64, kTrace>(a, s);
    case 128: return launch_hd<QT, OT, 128, kTrace>(a, s);
    case 256: return launch_hd<QT, OT, 256, kTrace>(a, s);
    default: return {};
  }
}

}  // namespace

// Blocks that the SMs hold at a time.
static int64_t places(int hd, int sms) {
  return (int64_t)sms * (hd == 64    ? Shape<64>::kBlocks
                         : hd == 128 ? Shape<128>::kBlocks
                                     : Shape<256>::kBlocks);
}

// Splits by the launch's sizes alone. A block costs about 3 us beside its tokens (128
// lanes of 128 to 4096 tokens, in row order: 108 us in splits of 4096, 117 of 1024, 138
// of 512), so the blocks of one lane are to fill two thirds of the places once: 131071
// tokens and 8 KV heads take 52 us in 38 splits (304 blocks, two an SM), 56 in 57 (456
// blocks on 456 places), 69 in 64, 68 in 256. Lanes differ in length and max_len is the
// longest, so several lanes aim at one and a half times the places (33 lanes of up to
// 3001 tokens, 2 heads of 256: 23 us in 3 splits, 33 in 2). No split is longer than 4096,
// so that one long lane among many is shared, or shorter than 256.
int attn_q8_split_len(int n, int Hkv, int hd, int max_len, int sms) {
  const int64_t room = places(hd, sms), pairs = std::max<int64_t>(1, (int64_t)n * Hkv);
  const int64_t want = n > 1 ? 3 * room / 2 : std::max<int64_t>(sms, 2 * room / 3);
  const int64_t splits = std::max<int64_t>(1, want / pairs);
  const int64_t len = (std::max(max_len, 1) + splits - 1) / splits;
  return (int)std::min<int64_t>(4096, std::max<int64_t>(256, (len + 127) / 128 * 128));
}

Launched launch_attention_q8(const AttnQ8& args, int q_type, int out_type, bool traced, int sms,
                             cudaStream_t s) {
  if (args.n <= 0) return {};
  AttnQ8 a = args;
  a.by_len = a.n <= kRankRows && a.max_len >= 2048 && a.split_len >= 2048 &&
             (int64_t)a.n * a.kv.Hkv >= 2 * places(a.kv.hd, sms);
  if (traced)
    return out_type == X_BF16 ? dispatch<float, __nv_bfloat16, true>(a, s)
                              : dispatch<float, float, true>(a, s);
  return out_type == X_BF16 ? dispatch<__nv_bfloat16, __nv_bfloat16, false>(a, s)
                            : dispatch<float, float, false>(a, s);
}

}  // namespace fsk
