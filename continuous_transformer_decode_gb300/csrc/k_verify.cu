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

#include <math_constants.h>

#include "fs_internal.h"

namespace fsk {
namespace {

constexpr int kT = 1024;

template <typename T, typename F>
__device__ T block_reduce(T v, T* sh, F f) {
  __syncthreads();
  sh[threadIdx.x] = v;
  __syncthreads();
  for (int w = kT / 2; w > 0; w >>= 1) {
    if (threadIdx.x < w) sh[threadIdx.x] = f(sh[threadIdx.x], sh[threadIdx.x + w]);
    __syncthreads();
  }
  return sh[0];
}

// weight of logit x under the row's largest logit m: exp((x - m) / T)
__device__ __forceinline__ double weight(float x, float m, double T) {
  return x == m ? 1.0 : (x > -CUDART_INF_F ? exp(((double)x - (double)m) / T) : 0.0);
}

__global__ void __launch_bounds__(kT) k_verify(VerifyArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ double sd[kT];
  __shared__ float sf[kT];
  __shared__ int si[kT];
  const int b = blockIdx.x, t = threadIdx.x, V = a.V;
  const int r0 = max(0, min(a.row_start[b], a.n_rows));
  const int r1 = max(r0, min(a.row_start[b + 1], a.n_rows));
  if (r0 == r1) {
    if (t == 0) {
      a.n_accepted[b] = 0;
      a.next_token[b] = -1;
    }
    return;
  }
  const float temp = a.temps[b];
  const int seg = (V + kT - 1) / kT, lo = min(V, t * seg), hi = min(V, lo + seg);
  for (int r = r0; r < r1; ++r) {
    const float* z = a.logits + r * a.ld_logits;
    const int x = a.draft[r];
    const bool last = r == r1 - 1, known = x >= 0 && x < V;
    float m = -CUDART_INF_F;
    for (int i = t; i < V; i += kT) m = fmaxf(m, z[i]);
    m = block_reduce(m, sf, [](float p, float q) { return fmaxf(p, q); });
    if (!(temp > 0.0f) || m == -CUDART_INF_F) {
      int best = V;
      for (int i = t; i < V; i += kT)
        if (z[i] == m) best = min(best, i);
      best = block_reduce(best, si, [](int p, int q) { return min(p, q); });
      if (m == -CUDART_INF_F) best = 0;  // no token at all: the sampler's answer
      if (!last && x == best && m > -CUDART_INF_F) continue;
      if (t == 0) {
        a.n_accepted[b] = r - r0;
        a.next_token[b] = best;
      }
      return;
    }
    const double T = temp;
    double S = 0.0;
    for (int i = t; i < V; i += kT) S += weight(z[i], m, T);
    S = block_reduce(S, sd, [](double p, double q) { return p + q; });
    if (!last && known) {
      const double q = a.probs ? (double)a.probs[r * a.ld_probs + x] : 1.0;
      if ((double)a.u_accept[r] * q * S < weight(z[x], m, T)) continue;
    }
    // what is left of p (times S)
    const float* pr = a.probs && !last ? a.probs + r * a.ld_probs : nullptr;
    auto left = [&](int i) {
      const double e = weight(z[i], m, T);
      if (pr) return fmax(e - (double)pr[i] * S, 0.0);
      return !last && !a.probs && i == x ? 0.0 : e;
    };
    double part = 0.0;
    for (int i = lo; i < hi; ++i) part += left(i);
    bool plain = !(block_reduce(part, sd, [](double p, double q) { return p + q; }) > 0.0);
    if (plain) {
      part = 0.0;
      for (int i = lo; i < hi; ++i) part += weight(z[i], m, T);
    }
    __syncthreads();
    sd[t] = part;
    __syncthreads();
    for (int w = 1; w < kT; w <<= 1) {
      const double v = t >= w ? sd[t - w] : 0.0;
      __syncthreads();
      sd[t] += v;
      __syncthreads();
    }
    const double target = (double)a.u_sample[b] * sd[kT - 1];
    int found = V, pos = -1;
    double cum = t ? sd[t - 1] : 0.0;
    for (int i = lo; i < hi; ++i) {
      const double e = plain ? weight(z[i], m, T) : left(i);
      cum += e;
      if (e > 0.0) {
        pos = i;
        if (cum >= target && found == V) found = i;
      }
    }
    found = block_reduce(found, si, [](int p, int q) { return min(p, q); });
    pos = block_reduce(pos, si, [](int p, int q) { return max(p, q); });
    if (t == 0) {
      a.n_accepted[b] = r - r0;
      a.next_token[b] = found < V ? found : pos;
    }
    return;
  }
}

}  // namespace

int launch_verify(const VerifyArgs& a, cudaStream_t s) {
  if (a.n_seqs <= 0) return 0;
  launch_k(k_verify, dim3(a.n_seqs), kT, 0, s, a);
  return 1;
}

}  // namespace fsk
