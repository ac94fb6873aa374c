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
// cluster serves a sequence: its blocks share a row's vocabulary, a warp a run
// of consecutive tokens, and exchange (max, sum) through distributed shared
// memory, one cluster barrier a row. The sum that decides an acceptance is in
// f32; where the decision comes within 2^-14 of its border (f32 sums of a
// vocabulary below a million are better than that) it is taken again from
// weights good to 2^-36, which also make the draw: its answer depends on the
// running sums of a whole row, and with f32 weights one draw in a few hundred
// would be another token. These weights and sums are pairs of f32 numbers: this
// GPU's f64 rate, 1/60 of its f32 rate, would bound the kernel.

#include <cooperative_groups.h>
#include <math_constants.h>

#include "fs_internal.h"
#include "two_f32.cuh"

namespace fsk {
namespace {

using namespace two;

namespace cg = cooperative_groups;

constexpr int kC = 8;        // blocks of a sequence's cluster
constexpr int kT = 512;      // threads of a block
constexpr int kW = kT / 32;  // warps of a block
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

// exp((z - m) / T) as 2^y, y = (z - m) * c with c = log2(e) / T, to a relative
// 2^-36: y = n + k/32 + f with |f| <= 1/64, 2^f = 1 + its Taylor series (the
// method of Tang, ACM TOMS 1989). Below 2^-126 it is zero.
__device__ __forceinline__ Two weight2(float z, float m, Two c, const float2* tab) {
  if (z == m) return {1.0f, 0.0f};
  const Two d = two_sum(z, -m);
  const float p = __fmul_rn(d.h, c.h);
  if (!(p > -125.5f)) return {0.0f, 0.0f};  // also -inf and NaN
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
  const float s = __int_as_float(((k >> 5) + 127) << 23);  // 2^n, -126 <= n <= 0
  return {__fmul_rn(r.h, s), __fmul_rn(r.l, s)};
}

// f32 weight under m; c = log2(e) / T.
__device__ __forceinline__ float weight1(float z, float m, float c) {
  return z == m ? 1.0f : z > -CUDART_INF_F ? exp2f((z - m) * c) : 0.0f;
}
// factor that takes sums under m to sums under M
__device__ __forceinline__ float rescale(float m, float M, float c) {
  return m == -CUDART_INF_F ? 0.0f : m == M ? 1.0f : exp2f((m - M) * c);
}

struct Stat {  // of a row's part
  float max, sum;  // sum of exp((z - max) / T)
  int best;        // lowest index of max
};

struct Shared {
  float2 tab[32];
  Stat warp[kW];
  Two wsum[kW];
  Stat part[2][kC];  // the cluster's blocks; two buffers, taken in turn: a block may
  Two psum[2][kC];   // write the next exchange while another still reads the last
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

// Every thread takes the decisions: they come from the same numbers in the same
// order in every block, so the cluster stays together.
__global__ void __launch_bounds__(kT) k_verify(VerifyArgs a) {
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid < 32) sh.tab[tid] = kExp2[tid];
  cluster.sync();  // every block has started: its shared memory can be written
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / kC, V = a.V;
  const int r0 = max(0, min(a.row_start[b], a.n_rows));
  const int r1 = max(r0, min(a.row_start[b + 1], a.n_rows));
  if (r0 == r1) {  // the whole cluster
    if (rank == 0 && tid == 0) {
      a.n_accepted[b] = 0;
      a.next_token[b] = -1;
    }
    return;
  }
  const float temp = a.temps[b];
  const bool greedy = !(temp > 0.0f);
  const Two c = log2e_over(greedy ? 1.0f : temp);
  // this warp's run of tokens [lo, hi)
  const int run = (V - 1) / (kC * kW * 128) * 128 + 128;
  const int lo = (int)min((int64_t)V, (int64_t)(rank * kW + warp) * run);
  const int hi = (int)min((int64_t)V, (int64_t)lo + run);
  int turn = 0;

  // the sum over the cluster, block by block in sh.psum[turn ^ 1] afterwards and
  // warp by warp in sh.wsum
  auto cluster_sum = [&](Two v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = add(v, shfl_xor(v, o));
    if (lane == 0) sh.wsum[warp] = v;
    __syncthreads();
    if (warp == 0) {
      v = lane < kW ? sh.wsum[lane] : Two{0.0f, 0.0f};
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v = add(v, shfl_xor(v, o));
      if (lane < kC) *cluster.map_shared_rank(&sh.psum[turn][rank], lane) = v;
    }
    cluster.sync();
    v = sh.psum[turn][0];
#pragma unroll
    for (int i = 1; i < kC; ++i) v = add(v, sh.psum[turn][i]);
    turn ^= 1;
    return v;
  };

  for (int r = r0; r < r1; ++r) {
    const float* z = a.logits + r * a.ld_logits;
    const bool vec = (reinterpret_cast<uintptr_t>(z) & 15) == 0;
    const bool last = r == r1 - 1;
    // ---- the row's maximum, its index, and its sum
    Stat st = {-CUDART_INF_F, 0.0f, V};
    {
      constexpr int kU = 4;  // groups of 128 tokens in flight
      for (int i0 = lo; i0 < hi; i0 += 128 * kU) {
        float4 v[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) v[u] = load4(z, i0 + 128 * u + 4 * lane, hi, vec);
        float mx = -CUDART_INF_F;
#pragma unroll
        for (int u = 0; u < kU; ++u)
          mx = fmaxf(mx, fmaxf(fmaxf(v[u].x, v[u].y), fmaxf(v[u].z, v[u].w)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, o));
        if (mx > st.max) st = {mx, st.sum * rescale(st.max, mx, c.h), V};
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const float x[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (greedy) {
              if (x[e] == mx && mx == st.max) st.best = min(st.best, i0 + 128 * u + 4 * lane + e);
            } else {
              st.sum += weight1(x[e], st.max, c.h);
            }
          }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        st.sum += __shfl_xor_sync(kAll, st.sum, o);
        st.best = min(st.best, __shfl_xor_sync(kAll, st.best, o));
      }
      // a run without a token: its -inf equal their maximum
      if (st.max == -CUDART_INF_F) st = {-CUDART_INF_F, 0.0f, V};
    }
    if (lane == 0) sh.warp[warp] = st;
    __syncthreads();
    if (warp == 0) {  // joins the warps; lane i writes block i's copy
      st = lane < kW ? sh.warp[lane] : Stat{-CUDART_INF_F, 0.0f, V};
      float M = st.max;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
      float sum = st.sum * rescale(st.max, M, c.h);
      int best = st.max == M ? st.best : V;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(kAll, sum, o);
        best = min(best, __shfl_xor_sync(kAll, best, o));
      }
      if (lane < kC) *cluster.map_shared_rank(&sh.part[turn][rank], lane) = {M, sum, best};
    }
    cluster.sync();
    float M = -CUDART_INF_F, S = 0.0f;
    int best = V;
#pragma unroll
    for (int i = 0; i < kC; ++i)
      if (sh.part[turn][i].max > M) {
        M = sh.part[turn][i].max;
        best = sh.part[turn][i].best;
      }
#pragma unroll
    for (int i = 0; i < kC; ++i)
      S += sh.part[turn][i].sum * rescale(sh.part[turn][i].max, M, c.h);
    turn ^= 1;
    // ---- greedy sequences, and rows without a token
    const int x = last ? -1 : a.draft[r];
    if (greedy || M == -CUDART_INF_F) {
      if (M == -CUDART_INF_F) best = 0;
      if (!last && x == best && M > -CUDART_INF_F) continue;
      if (rank == 0 && tid == 0) {
        a.n_accepted[b] = r - r0;
        a.next_token[b] = best;
      }
      break;
    }
    // ---- accept?
    Two S2 = {0.0f, 0.0f};  // the sum to 2^-36, once it is needed
    auto precise_sum = [&]() {
      Two s = {0.0f, 0.0f};
      for (int i = lo + 4 * lane; i < hi; i += 128) {
        const float4 v = load4(z, i, hi, vec);
        s = add(s, add(add(weight2(v.x, M, c, sh.tab), weight2(v.y, M, c, sh.tab)),
                       add(weight2(v.z, M, c, sh.tab), weight2(v.w, M, c, sh.tab))));
      }
      return cluster_sum(s);
    };
    if (!last && x >= 0 && x < V) {
      const float u = a.u_accept[r], q = a.probs ? a.probs[r * a.ld_probs + x] : 1.0f;
      const Two w = weight2(z[x], M, c, sh.tab);
      const float t = u * q * S;
      bool ok = t < w.h;
      if (fabsf(t - w.h) <= 0x1p-14f * w.h) {
        S2 = precise_sum();
        ok = less(mul(mul({u, 0.0f}, {q, 0.0f}), S2), w);
      }
      if (ok) continue;
    }
    // ---- the draw
    const float* pr = a.probs && !last ? a.probs + r * a.ld_probs : nullptr;
    const bool pvec = pr && (reinterpret_cast<uintptr_t>(pr) & 15) == 0;
    if (pr && S2.h == 0.0f) S2 = precise_sum();
    bool minus = pr != nullptr;          // the draft's probabilities are taken off
    int out = minus || last ? -1 : x;    // the token that is taken out
    // what is left of four tokens: weight e and draft probability q give max(e - q S, 0)
    auto left4 = [&](int i, Two o[4]) {
      const float4 v = load4(z, i, hi, vec);
      float4 q4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (minus) q4 = load4(pr, i, hi, pvec);
      const float zz[4] = {v.x, v.y, v.z, v.w}, q[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[j] = weight2(zz[j], M, c, sh.tab);
        if (i + j == out) o[j] = {0.0f, 0.0f};
        if (minus && o[j].h > 0.0f) {
          const Two p = mul({q[j], 0.0f}, S2);
          o[j] = add(o[j], {-p.h, -p.l});
          if (!(o[j].h > 0.0f)) o[j] = {0.0f, 0.0f};
        }
      }
    };
    Two total;
    for (int attempt = 0; attempt < 2; ++attempt) {
      Two s = {0.0f, 0.0f};
      for (int i = lo + 4 * lane; i < hi; i += 128) {
        Two o[4];
        left4(i, o);
        s = add(s, add(add(o[0], o[1]), add(o[2], o[3])));
      }
      total = cluster_sum(s);
      if (total.h > 0.0f) break;
      minus = false;  // nothing is left: from p itself
      out = -1;
    }
    const Two target = mul({fminf(a.u_sample[b], 1.0f), 0.0f}, total);
    // the first of `n` parts with a weight whose running sum reaches the target
    // (the last with a weight, should rounding leave the target above the total)
    auto pick = [&](const Two* part, int n, Two& before) {
      int at = -1;
      for (int i = 0; i < n; ++i) {
        if (!(part[i].h > 0.0f)) continue;
        if (at >= 0) {
          const Two upto = add(before, part[at]);
          if (!less(upto, target)) break;
          before = upto;
        }
        at = i;
      }
      return at;
    };
    Two cum = {0.0f, 0.0f};
    if (pick(sh.psum[turn ^ 1], kC, cum) == rank && pick(sh.wsum, kW, cum) == warp) {
      int found = V, pos = -1;
      for (int i0 = lo; i0 < hi && !__any_sync(kAll, found < V); i0 += 128) {
        const int i = i0 + 4 * lane;
        Two o[4];
        left4(i, o);
        const Two s = add(add(o[0], o[1]), add(o[2], o[3]));
        Two at = s;  // inclusive scan over the lanes, then exclusive
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const Two up = {__shfl_up_sync(kAll, at.h, d), __shfl_up_sync(kAll, at.l, d)};
          if (lane >= d) at = add(up, at);
        }
        const Two end = add(cum, {__shfl_sync(kAll, at.h, 31), __shfl_sync(kAll, at.l, 31)});
        at = {__shfl_up_sync(kAll, at.h, 1), __shfl_up_sync(kAll, at.l, 1)};
        at = lane ? add(cum, at) : cum;
        cum = end;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          at = add(at, o[j]);
          if (o[j].h > 0.0f) {
            pos = i + j;
            if (!less(at, target)) found = min(found, i + j);
          }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        found = min(found, __shfl_xor_sync(kAll, found, o));
        pos = max(pos, __shfl_xor_sync(kAll, pos, o));
      }
      if (lane == 0) {
        a.n_accepted[b] = r - r0;
        a.next_token[b] = found < V ? found : pos;
      }
    }
    break;
  }
  cluster.sync();  // no block leaves while another may still write to it
}

}  // namespace

int launch_verify(const VerifyArgs& a, cudaStream_t s) {
  if (a.n_seqs <= 0) return 0;
  launch_k_cluster(k_verify, dim3((unsigned)a.n_seqs * kC), kT, 0, s, kC, a);
  return 1;
}

}  // namespace fsk
