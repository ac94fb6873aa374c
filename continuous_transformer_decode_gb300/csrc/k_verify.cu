// Verification of drafted tokens: speculative sampling's accept / resample
// rule over the target's logits (Leviathan et al., ICML 2023), from random
// numbers that the caller gives.
//
// Row r of a sequence holds the target's logits z after which the draft
// proposed x = draft[r] with probability q(x). With p = softmax(z / T), x is
// accepted while u_accept[r] * q(x) < p(x); the first row whose token is not
// gives the next token from max(p - q, 0), or, when all are accepted, the
// last row from p: the first index whose running sum reaches
// u_sample * total.
//
// The bytes are the rows of logits, each wanted once. A sequence's rows are
// taken in order and those after a rejection are never read. One thread-block
// cluster serves a sequence: its warps share a row's vocabulary in runs of
// consecutive tokens, and each writes its (max, sum) into every block's shared
// memory: one cluster barrier a row, and one more for a draw.
//
// Whole-number answers are held to more than f32: where an acceptance or a draw
// comes so near to its border that f32 weights and sums cannot tell, it is taken
// again from weights good to 2^-36, as pairs of f32 numbers (this GPU's f64 rate is
// 1/60 of its f32 rate). What f32 may be off by is derived, not measured (in the kernel,
// below). That is rare for an acceptance, and 10 to 13 draws in a hundred for normal
// logits over a vocabulary of 32000 to 49152. What bounds the kernel is the chain of one
// sequence on eight SMs (2 to 3 us a row: a row's loads, its maximum and sum, the
// barrier; and 9 us for a draw that is taken again with draft probabilities), not the
// bytes. Means over many inputs: 256 sequences of 4 drafts from a lookup, 49152 tokens,
// 37 us, 61 to 77 MB of logits being read (every draw taken again: 61 us); 64 sequences
// of 0 to 7 drafts 35 us (45 us); one of 4 drafts 11 us (19 us).

#include <cooperative_groups.h>
#include <math_constants.h>

#include "fs_internal.h"
#include "two_f32.cuh"

namespace fsk {
namespace {

using namespace two;

namespace cg = cooperative_groups;

constexpr unsigned kAll = 0xffffffffu;

// 2^(k/32) as pairs of f32 numbers.
__constant__ float2 kExp2[32] = {
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

struct Stat {  // of a row's part
  float max, sum;  // sum of exp((z - max) / T)
  int best;        // lowest index of max
};

// Every warp of the cluster writes what it found to all blocks; two buffers, taken in
// turn: a block may write the next exchange while another still reads the last.
template <int kC, int kW>
struct Shared {
  float2 tab[32];
  Stat stat[2][kC * kW];
  Two sum[2][kC * kW];
  float scan[kW];
  Two scan2[kW];
  int at[kW], tail[kW];
  int again;  // the f32 draw could not tell
};

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

// What is left of the block's tokens for the draw, in pairs: weight e; with draft
// probabilities max(e - q S, 0); without token `out`.
struct Left {
  const float* z;
  const float* q;  // null: none
  float M;
  Two c, S;
  int out;
  const float2* tab;
  template <bool kQ>
  __device__ __forceinline__ Two at(int i) const {
    const Two e = weight2(z[i], M, c, tab);
    if constexpr (!kQ) return {i == out ? 0.0f : e.h, i == out ? 0.0f : e.l};
    const Two p = mul({q[i], 0.0f}, S), d = add(e, {-p.h, -p.l});
    const bool some = e.h > 0.0f && d.h > 0.0f;
    return {some ? d.h : 0.0f, some ? d.l : 0.0f};
  }
  __device__ __forceinline__ Two at(int i) const { return q ? at<true>(i) : at<false>(i); }
};
// A lane's share of tokens lo .. hi - 1, four at a time for their latencies. Out of
// line: it runs seldom, from several places.
template <bool kQ>
__device__ __noinline__ Two left_sum_of(Left w, int lo, int hi, int lane) {
  Two s[4] = {};
#pragma unroll 1
  for (int i = lo + lane; i < hi; i += 128) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int j = min(i + 32 * u, hi - 1);  // all four in step, those past the end unused
      const Two e = w.at<kQ>(j);
      const bool in = i + 32 * u < hi;
      s[u] = add(s[u], {in ? e.h : 0.0f, in ? e.l : 0.0f});
    }
  }
  return add(add(s[0], s[1]), add(s[2], s[3]));
}
__device__ __forceinline__ Two left_sum(const Left& w, int lo, int hi, int lane) {
  return w.q ? left_sum_of<true>(w, lo, hi, lane) : left_sum_of<false>(w, lo, hi, lane);
}

// Every thread takes the decisions: they come from the same numbers in the same
// order in every block, so the cluster stays together.
//
// held: a block's part of the row (and of the draft's probabilities) stays in
// dynamic shared memory for the draw; else it is read again. Three blocks an SM, which is
// 80 registers (left to itself the compiler takes up to 93, and 256 sequences 12 % longer).
template <int kC, int kT>
__global__ void __launch_bounds__(kT, 3) k_verify(VerifyArgs a, int held) {
  constexpr int kW = kT / 32;
  __shared__ Shared<kC, kW> sh;
  extern __shared__ __align__(16) float hold[];  // [kW * run] z, then q
  cg::cluster_group cluster = cg::this_cluster();
  auto sync = [&] {
    if constexpr (kC == 1) __syncthreads();
    else cluster.sync();
  };
  auto remote = [&](auto* p, int r) {
    if constexpr (kC == 1) return p;
    else return cluster.map_shared_rank(p, r);
  };
  const int rank = kC == 1 ? 0 : (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < 32) sh.tab[tid] = kExp2[tid];
  if (tid == 0) sh.again = 0;
  // the other blocks' shared memory can be written once they have started: arrive
  // now, wait before the first write
  if constexpr (kC > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  auto started = [&] {
    if constexpr (kC > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  };
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / kC, V = a.V;
  const int first = a.row_start[b], end = a.row_start[b + 1];
  const float temp = a.temps[b], us = fminf(a.u_sample[b], 1.0f);
  const int r0 = max(0, min(first, a.n_rows)), r1 = max(r0, min(end, a.n_rows));
  if (r0 == r1) {  // the whole cluster
    if (rank == 0 && tid == 0) {
      a.n_accepted[b] = 0;
      a.next_token[b] = -1;
    }
    started();
    return;
  }
  const bool greedy = !(temp > 0.0f);
  // outside this range only the largest logits count, or all alike
  const Two c = log2e_over(greedy ? 1.0f : fminf(fmaxf(temp, 1e-30f), 1e30f));
  // this block's tokens are base .. base + count - 1, this warp's lo .. hi - 1 of them
  const int run = (V - 1) / (kC * kW * 128) * 128 + 128;
  const int base = (int)min((int64_t)V, (int64_t)rank * kW * run);
  const int count = (int)min((int64_t)V - base, (int64_t)kW * run);
  const int lo = min(count, warp * run), hi = min(count, lo + run);
  // How far f32 may be off, in units of 2^-24. A weight: 4 + 1.4 |y| (weight1). A lane
  // sums sixteen weights of a chunk in five additions that round, and chunk by chunk
  // takes its sum to a new maximum (a product by a weight, 5 + 1.4 |y|) and adds, 6 a
  // chunk; five more sum the lanes, one product takes a warp's sum to the row's maximum
  // and six additions sum the warps. The |y| of a token's weight and of the factors
  // that it meets add up to its |y| under the row's maximum, and the mean of that over
  // the row is log2(V / S) at most, as -sum p log2 p <= log2 V. So S is off by
  // 25 + 6 chunks + 1.4 log2(V / S).
  //
  // In a draw, an error that a running sum P and the total share moves P - u total by
  // max(u, 1 - u) of itself at most. So, of S: the warps' sums, 19 + 6 chunks +
  // 1.4 log2(V / S); the additions that give the total and the running sum, and the
  // product by u, 15; 6 of a weight of 1 for the draft's, taken out (5 + 1.4 |y| of it).
  // The chosen warp's tokens are summed anew: their weights, with a mean |y| of
  // log2(run / own) if own is their sum, and additions of numbers up to own, ten of the
  // scans, four for the place and two a chunk. With draft probabilities a weight
  // max(e - q S, 0) is off by e (5 + 1.4 |y|) and, where it is not zero, S's error times e,
  // and they are summed in 7 + 4 chunks additions. (Weights of equal logits err alike, so
  // nothing is taken to cancel: what suffices where roundings are independent, 6 or 8 of
  // S in all, gave wrong tokens in rows of 262144.)
  const float log_run = lg2((float)run);
  const float chunks = (float)((run + 511) / 512), log_v = lg2((float)V);
  constexpr float kUnit = 0x1p-24f;
  int turn = 0;
  constexpr int kN = kC * kW;  // warps of the cluster, two a lane in what follows
  static_assert(kN <= 64, "two warps a lane");
  const int e0 = 2 * lane, e1 = 2 * lane + 1;
  // the sum of the lanes' v over the cluster; the warps' sums are in w0 and w1
  Two w0, w1;
  auto cluster_sum = [&](Two v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = add(v, shfl_xor(v, o));
    if (lane < kC) *remote(&sh.sum[turn][rank * kW + warp], lane) = v;
    sync();
    w0 = e0 < kN ? sh.sum[turn][e0] : Two{0.0f, 0.0f};
    w1 = e1 < kN ? sh.sum[turn][e1] : Two{0.0f, 0.0f};
    turn ^= 1;
    v = add(w0, w1);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = add(v, shfl_xor(v, o));
    return v;
  };

  // chunks of kU groups of 128 tokens, the next one on its way while one is worked
  // on; after a row's last comes the first of the next row, which is wanted if the
  // draft is accepted
  constexpr int kU = 4;
  float4 next[kU];
  auto fetch = [&](int row, int i0) {
    const float* z = a.logits + row * a.ld_logits + base;
    const bool vec = (reinterpret_cast<uintptr_t>(z) & 15) == 0;
#pragma unroll
    for (int u = 0; u < kU; ++u) next[u] = load4(z, i0 + 128 * u + 4 * lane, hi, vec);
  };
  fetch(r0, lo);
#pragma unroll 1
  for (int r = r0; r < r1; ++r) {
    const float* z = a.logits + r * a.ld_logits + base;
    const bool last = r == r1 - 1;
    // what decides on the draft
    const int x = last ? -1 : a.draft[r];
    const bool known = x >= 0 && x < V;
    const float u_acc = known ? a.u_accept[r] : 0.0f, z_x = known ? z[x - base] : 0.0f;
    const float q_x = known && a.probs ? a.probs[r * a.ld_probs + x] : 1.0f;
    // ---- the row's maximum, its index, and its sum
    Stat st = {-CUDART_INF_F, 0.0f, V};
#pragma unroll 1
    for (int i0 = lo; i0 < hi; i0 += 128 * kU) {
      float4 v[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) v[u] = next[u];
      const bool more = i0 + 128 * kU < hi;
      if (more || !last) fetch(more ? r : r + 1, more ? i0 + 128 * kU : lo);
      if (held)
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (i0 + 128 * u < lo + run)
            *reinterpret_cast<float4*>(hold + i0 + 128 * u + 4 * lane) = v[u];
      float mx = -CUDART_INF_F;
#pragma unroll
      for (int u = 0; u < kU; ++u)
        mx = fmaxf(mx, fmaxf(fmaxf(v[u].x, v[u].y), fmaxf(v[u].z, v[u].w)));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, o));
      if (mx > st.max) st = {mx, st.sum * rescale(st.max, mx, c), V};
      if (greedy) {
        if (mx == st.max && st.best == V) {
#pragma unroll
          for (int u = kU - 1; u >= 0; --u) {
            const int i = base + i0 + 128 * u + 4 * lane;
            if (v[u].w == mx) st.best = i + 3;
            if (v[u].z == mx) st.best = i + 2;
            if (v[u].y == mx) st.best = i + 1;
            if (v[u].x == mx) st.best = i;
          }
        }
      } else {
        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          part[0] += weight1(v[u].x, st.max, c);
          part[1] += weight1(v[u].y, st.max, c);
          part[2] += weight1(v[u].z, st.max, c);
          part[3] += weight1(v[u].w, st.max, c);
        }
        st.sum += (part[0] + part[1]) + (part[2] + part[3]);
      }
    }
    if (greedy) {
      st.best = __reduce_min_sync(kAll, st.best);
    } else {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) st.sum += __shfl_xor_sync(kAll, st.sum, o);
    }
    // a run without a token: its -inf equal their maximum
    if (st.max == -CUDART_INF_F) st = {-CUDART_INF_F, 0.0f, V};
    if (r == r0) started();
    if (lane < kC) *remote(&sh.stat[turn][rank * kW + warp], lane) = st;
    sync();
    const Stat none = {-CUDART_INF_F, 0.0f, V};
    const Stat s0 = e0 < kN ? sh.stat[turn][e0] : none, s1 = e1 < kN ? sh.stat[turn][e1] : none;
    turn ^= 1;
    float M = fmaxf(s0.max, s1.max);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
    // ---- greedy sequences, and rows without a token
    if (greedy || M == -CUDART_INF_F) {
      int best = __reduce_min_sync(kAll, s0.max == M ? s0.best : s1.max == M ? s1.best : V);
      if (M == -CUDART_INF_F) best = 0;
      if (!last && x == best && M > -CUDART_INF_F) continue;
      if (rank == 0 && tid == 0) {
        a.n_accepted[b] = r - r0;
        a.next_token[b] = best;
      }
      break;
    }
    // the warps' sums under M, and the row's
    float f0 = s0.sum * rescale(s0.max, M, c), f1 = s1.sum * rescale(s1.max, M, c), S = f0 + f1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) S += __shfl_xor_sync(kAll, S, o);
    // ---- accept?
    Left left = {held ? hold : z, nullptr, M, c, {0.0f, 0.0f}, -1, sh.tab};
    float wx = 0.0f;  // the weight of the draft
    if (known) {
      wx = weight1(z_x, M, c);
      const float t = u_acc * S * q_x;
      bool ok = t < wx;
      // t is off by S's error and two products, wx by a weight's, and two units are for
      // the products of errors. Below 2^-100 t's products may leave f32's range.
      const float deep = z_x == M ? 0.0f : fabsf(z_x - M) * c.h;
      const float unsure = 33.0f + 6.0f * chunks + 1.4f * (log_v - lg2(S) + deep);
      if (wx > 0.0f && (wx < 0x1p-100f || fabsf(t - wx) <= unsure * kUnit * wx)) {
        const Two S2 = cluster_sum(left_sum(left, lo, hi, lane));
        ok = less(mul(mul({u_acc, 0.0f}, S2), {q_x, 0.0f}), weight2(z_x, M, c, sh.tab));
      }
      if (ok) continue;
    }
    // ---- the draw, first in f32. Weights are e, or max(e - q S, 0), or e without x.
    const float* pr = a.probs && !last ? a.probs + r * a.ld_probs + base : nullptr;
    const bool takes = known && !a.probs;
    const int gone = takes ? x - base : -1;  // the token that is taken out, if it is here
    float* const hold_q = hold + kW * run;
    if (pr) {
      const bool pvec = (reinterpret_cast<uintptr_t>(pr) & 15) == 0;
      const bool zvec = (reinterpret_cast<uintptr_t>(z) & 15) == 0;
      float s = 0.0f;
#pragma unroll 1
      for (int i0 = lo; i0 < hi; i0 += 128 * kU) {
        float4 q[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) q[u] = load4(pr, i0 + 128 * u + 4 * lane, hi, pvec);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const int i = i0 + 128 * u + 4 * lane;
          if (i >= hi) continue;  // past the end z and q are -inf
          float4 v;
          if (held) {
            *reinterpret_cast<float4*>(hold_q + i) = q[u];
            v = *reinterpret_cast<const float4*>(hold + i);
          } else {
            v = load4(z, i, hi, zvec);
          }
          const float e0 = weight1(v.x, M, c), e1 = weight1(v.y, M, c);
          const float e2 = weight1(v.z, M, c), e3 = weight1(v.w, M, c);
          s += (e0 > 0.0f ? fmaxf(fmaf(-q[u].x, S, e0), 0.0f) : 0.0f) +
               (e1 > 0.0f ? fmaxf(fmaf(-q[u].y, S, e1), 0.0f) : 0.0f) +
               ((e2 > 0.0f ? fmaxf(fmaf(-q[u].z, S, e2), 0.0f) : 0.0f) +
                (e3 > 0.0f ? fmaxf(fmaf(-q[u].w, S, e3), 0.0f) : 0.0f));
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
      float* const sums = reinterpret_cast<float*>(sh.sum[turn]);
      if (lane < kC) *remote(sums + rank * kW + warp, lane) = s;
      sync();
      f0 = e0 < kN ? sums[e0] : 0.0f;
      f1 = e1 < kN ? sums[e1] : 0.0f;
      turn ^= 1;
    } else if (takes) {  // the warps' weights are known from the row's sum
      if (x / run == e0) f0 -= wx;
      if (x / run == e1) f1 -= wx;
    }
    const float* zs = held ? hold : z;
    const float* qs = !pr ? nullptr : held ? hold_q : pr;
    float total = f0 + f1, before = 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
    const float target = us * total;
    const int chosen = pick(f0, f1, target, before, lane);
    if (chosen >= 0 && chosen / kW == rank) {
      const int w = chosen % kW;
      const int end_w = min(count, (w + 1) * run);
      // what the running sum is ahead of the target, and what that may be off by
      float place = before - target;
      const float own = fmaxf(__shfl_sync(kAll, chosen & 1 ? f1 : f0, chosen / 2), 0x1p-100f);
      const float log_row = log_v - lg2(S);
      const float row = pr ? 52.0f + 10.0f * chunks + 2.8f * log_row
                           : 34.0f + 6.0f * chunks + 1.4f * log_row;
      const float off = kUnit * (row * S + 6.0f +
                                 (18.0f + 2.0f * chunks + 1.4f * (log_run - lg2(own))) * own);
      bool hit = false;  // a token whose borders the target is clear of
#pragma unroll 1
      for (int i0 = w * run; i0 < end_w; i0 += kT) {  // a token a thread
        const int i = i0 + tid;
        float e = i < end_w && i != gone ? weight1(zs[i], M, c) : 0.0f;
        if (qs && e > 0.0f) e = fmaxf(fmaf(-qs[i], S, e), 0.0f);
        const float inc = scan(e, lane);
        if (lane == 31) sh.scan[warp] = inc;
        __syncthreads();
        const float in_warps = scan(lane < kW ? sh.scan[lane] : 0.0f, lane);
        const float ahead = warp ? __shfl_sync(kAll, in_warps, warp - 1) : 0.0f;
        const float at = place + ahead + (inc - e), then = place + ahead + inc;
        const bool mine = at + off < 0.0f && 0.0f <= then - off;
        if (mine) {
          a.n_accepted[b] = r - r0;
          a.next_token[b] = base + i;
        }
        place += __shfl_sync(kAll, in_warps, 31);
        hit = __syncthreads_or(mine);
        if (hit || place >= off) break;
      }
      if (!hit && tid < kC) *remote(&sh.again, tid) = 1;
    }
    // a total of nothing, or of NaN: every block sees it
    if (!(total > 0.0f && chosen >= 0) && tid == 0) sh.again = 1;
    sync();  // also: no block leaves while another may still write to it
    if (!sh.again) return;
    // ---- the draw again, in pairs
    if (pr) {
      left.S = cluster_sum(left_sum(left, lo, hi, lane));
      left.q = qs;
    }
    left.out = gone;
    Two sum = cluster_sum(left_sum(left, lo, hi, lane));
    if (!(sum.h > 0.0f)) {  // nothing is left: from p itself
      left.q = nullptr;
      left.out = -1;
      sum = cluster_sum(left_sum(left, lo, hi, lane));
    }
    const Two goal = mul({us, 0.0f}, sum);
    Two cum = {0.0f, 0.0f};
    const int taken = pick(w0, w1, goal, cum, lane);
    if (taken >= 0 && taken / kW == rank) {
      // its run in the warps' lanes, `each` consecutive tokens a lane
      const int from = taken % kW * run, upto = min(count, from + run);
      const int each = (run + kT - 1) / kT, mine = from + tid * each;
      Two e = {0.0f, 0.0f};
      int tail = -1;
#pragma unroll 4
      for (int i = mine; i < min(upto, mine + each); ++i) {
        const Two v = left.at(i);
        if (v.h > 0.0f) tail = i;
        e = add(e, v);
      }
      Two at = scan(e, lane);
      if (lane == 31) sh.scan2[warp] = at;
      __syncthreads();
      const Two in_warps = scan(lane < kW ? sh.scan2[lane] : Two{0.0f, 0.0f}, lane);
      if (warp) cum = add(cum, shfl(in_warps, warp - 1));
      // the first lane that reaches the goal looks for its first token that does; the
      // run's last token with a weight is taken if none does
      const unsigned m = __ballot_sync(kAll, e.h > 0.0f && !less(add(cum, at), goal));
      tail = __reduce_max_sync(kAll, tail);
      if (lane == 0) sh.at[warp] = V, sh.tail[warp] = tail;
      __syncwarp();
      if (m) {
        const int who = __ffs(m) - 1, start = mine + (who - lane) * each;
        if (who) cum = add(cum, shfl(at, who - 1));
        int found = -1, last_in = -1;
        for (int i0 = start; i0 < min(upto, start + each) && found < 0; i0 += 32) {
          const int i = i0 + lane;
          const Two v = i < min(upto, start + each) ? left.at(i) : Two{0.0f, 0.0f};
          const Two s = add(cum, scan(v, lane));
          const unsigned h = __ballot_sync(kAll, v.h > 0.0f);
          const unsigned r = __ballot_sync(kAll, v.h > 0.0f && !less(s, goal));
          cum = shfl(s, 31);
          if (r) found = i0 + __ffs(r) - 1;
          if (h) last_in = i0 + 31 - __clz(h);
        }
        if (lane == 0) sh.at[warp] = found >= 0 ? found : last_in;
      }
      __syncthreads();
      const int lowest = __reduce_min_sync(kAll, lane < kW ? sh.at[lane] : V);
      const int highest = __reduce_max_sync(kAll, lane < kW ? sh.tail[lane] : -1);
      if (tid == 0) {
        a.n_accepted[b] = r - r0;
        a.next_token[b] = base + (lowest < V ? lowest : highest);
      }
    }
    break;
  }
  sync();  // no block leaves while another may still write to it
}

template <int kC>
Launched launch_c(const VerifyArgs& a, cudaStream_t s) {
  constexpr int kT = 256, kW = kT / 32;
  constexpr int64_t kMost = 56 * 1024;  // shared memory of four blocks an SM
  const int64_t run = (a.V - 1) / (kC * kW * 128) * 128 + 128;
  int64_t smem = kW * run * 4 * (a.probs ? 2 : 1);
  const int held = smem <= kMost;
  if (!held) smem = 0;
  static std::atomic<uint64_t> done{0};
  Launched l;
  l.error = allow_smem(k_verify<kC, kT>, (int)kMost, done);
  if (l.error != cudaSuccess) return l;
  if constexpr (kC == 1)
    l.add(launch_k(k_verify<1, kT>, dim3((unsigned)a.n_seqs), kT, smem, s, a, held));
  else
    l.add(launch_k_cluster(k_verify<kC, kT>, dim3((unsigned)a.n_seqs * kC), kT, smem, s, kC, a, held));
  return l;
}

}  // namespace

// Blocks of a sequence: eight while all sequences' blocks fit the SMs four at a time,
// else four (64 sequences: 35 us with eight, 58 with four; 256: 47 and 37), and no more
// than give every warp 128 tokens.
Launched launch_verify(const VerifyArgs& a, int sms, cudaStream_t s) {
  if (a.n_seqs <= 0) return {};
  const int want = (int64_t)a.n_seqs * 8 <= 4 * (int64_t)sms ? 8 : 4;
  if (a.V > 4096 && want == 8) return launch_c<8>(a, s);
  if (a.V > 2048) return launch_c<4>(a, s);
  return a.V > 1024 ? launch_c<2>(a, s) : launch_c<1>(a, s);
}

}  // namespace fsk
