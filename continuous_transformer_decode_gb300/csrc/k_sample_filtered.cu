// Sampling with temperature, top-k, top-p and min-p from given random numbers
// (fs_sample_filtered).
//
// With tokens ranked by (logit descending, index ascending), what top-k and top-p keep is a
// prefix of the ranking: all that is wanted is its last token, the cut. Nothing is sorted.
// A cut is found by counting: tokens fall into bins of y = (max - z) log2(e) / T (a weight
// is 2^-y), the bin in which the running count or mass passes the target is split again,
// and once few enough tokens are left they are ranked among themselves.
//
// Whole-number answers need more than f32 (a cut lies between tokens whose weights are
// 1e-6 of the sum): weights are whole numbers of 2^-39 of their bin's largest, good to
// 2^-38, and their sums do not depend on the order; sums of bins, and a draw's running sums,
// are pairs of f32 numbers. (f64 runs at 1/60 of f32's rate here.)
//
// A block or a cluster of two, four or eight serves a row and reads it once, into shared memory
// (the choice and its times are at launch_sample_filtered). A thread has a run of consecutive
// tokens and a column of the bins' counts and masses for itself (no atomics). What the draw
// needs, the kept mass of each run in order, is then the sum of a column's bins ahead of the
// cut; only the tokens of the cut's own bin are weighed again. They are gathered first (a tenth
// of the tokens, in lanes of their own), as the split and the ranking want them as well. Where
// the tokens up to the cut are few, as with a small top_k or a peaked row, they go to one block
// as a whole, which does the rest; a small top_k asks for no weights but theirs. Where min-p
// certainly ends ahead of the cut's bin, the cut is not looked for.
//
// The logits' bytes are a few percent of the time (256 rows of 49152: 7 us at the copy's rate).
// A row's chain bounds it, and the issue slots, half of them used: 256 rows with top-p take
// four waves of two blocks a row, 104 us, 47 of them the issue of 56 million instructions (66 for
// each token's weight); the rest is what 16 warps an SM wait for, barriers, shared memory and
// each other. 64 mixed rows: 32 us; one row of 32000 with top-k 50 and top-p: 10 us.

#include <cooperative_groups.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "draw.cuh"
#include "fs_internal.h"

namespace fsk {
namespace {

using namespace draw;

namespace cg = cooperative_groups;

// Bins of y: (b - 1, b], the last one also all above. Two more where a row has few blocks, whose
// shared memory has room for them: more cuts have room for their tokens behind them (64 rows of
// 49152, T = 1, top-p 0.998: 31 us, 42 with 20 bins; 0.95: 29.3 and 29.0).
template <int kC>
constexpr int kBinsOf = kC < 4 ? 22 : 20;
constexpr int kSub = 64;    // parts of a bin that is split
constexpr int kList = 128;  // tokens that are ranked among themselves
constexpr int kFew = 64;    // a top_k that always ends in one list
constexpr int kFrac = 39;   // a mass in bin b is a whole number of 2^-(b + kFrac)
constexpr int kLeast = -125 * 256;  // weights at this place and behind are 0
constexpr int kCount = 50;  // a column's entry: count << kCount | mass

struct Bin {
  uint64_t mass;
  uint32_t count, pad;
};
struct Kept {
  Two mass;
  int count;
};
struct Power {  // 2^(k/256): times 2^kFrac, and as a pair
  uint64_t whole;
  float h, l;
};

template <int kC, int kW>
struct Shared {
  Power tab[256];
  float max[kC * kW];
  int at[kC * kW];
  Kept kept[kC * kW];
  Bin bins[kC][kBinsOf<kC>];
  Bin sub[kC][kSub];
  uint32_t own[3 + 1][kSub];  // of this block: a mass in three, and the count
  uint64_t range[kC][2];
  unsigned long long lo, hi;
  uint64_t list[2][kList], sorted[kList];
  Two scan[kW];
  int hit, fill, taken;
  struct {  // what one warp found for all
    Two before;
    uint32_t ahead, left;
    int at;
  } found;
};

__device__ __forceinline__ Two to_two(uint64_t m, int e) {  // m * 2^e, -127 < e < 87
  const float s = __int_as_float((127 + e) << 23);
  const float h = (float)(uint32_t)(m >> 40) * 0x1p40f, i = (float)((uint32_t)(m >> 20) & 0xfffffu) * 0x1p20f;
  const Two t = fast_two_sum(h, i);
  const Two u = fast_two_sum(t.h, __fadd_rn(t.l, (float)((uint32_t)m & 0xfffffu)));
  return {u.h * s, u.l * s};
}

// The rank of a token, the first the smallest: its logit's bits in falling order, then
// its index.
__device__ __forceinline__ uint64_t rank_of(float z, int i) {
  const uint32_t u = __float_as_uint(z);
  const uint32_t falling = (u >> 31) ? u : ~(u | 0x80000000u);
  return ((uint64_t)falling << 32) | (uint32_t)i;
}
__device__ __forceinline__ float logit_of(uint64_t r) {
  const uint32_t f = (uint32_t)(r >> 32);
  return __uint_as_float((f >> 31) ? f : (~f & 0x7fffffffu));
}

// -0 as 0 and NaN as -inf.
__device__ __forceinline__ float clean(float z) { return fmaxf(z, -CUDART_INF_F) + 0.0f; }

// The largest of the lanes' values (no NaN, no -0).
__device__ __forceinline__ float warp_max(float v) {
  const int i = __float_as_int(v);
  const int m = __reduce_max_sync(kAll, i ^ ((i >> 31) & 0x7fffffff));
  return __int_as_float(m ^ ((m >> 31) & 0x7fffffff));
}

// -256 y of a logit, rounded to a whole number: 0 for M (also an infinite one), at least
// -126 * 256. It falls with the logit; bins and their parts are ranges of it.
constexpr float kRound = 49152.0f;  // numbers of its size have 1/256 as their last place
__device__ __forceinline__ float to_grid(float p) { return __fadd_rn(fmaxf(fminf(p, 0.0f), -126.0f), kRound); }
__device__ __forceinline__ int steps_of(float t) { return __float_as_int(t) - __float_as_int(kRound); }
__device__ __forceinline__ int place(float z, float M, Two c) {
  return steps_of(to_grid(__fmul_rn(__fadd_rn(z, -M), c.h)));
}
// Of kSub parts of a bin, the last one apart.
__device__ __forceinline__ int part_of(int k, int y) { return (255 - k - 256 * y) >> 2; }
static_assert(kSub == 64, "four of 256 steps");

// exp((z - M) / T) = m 2^(n - kFrac), 2^kFrac <= m <= 2^(kFrac + 1); c = log2(e) / T. With y
// as a pair, k = place(z) and f the rest, 2^f - 1 is its Taylor series (the f^4 term is below
// 2^-42) and 2^(k/256) comes from the table: Tang's method (ACM TOMS 1989). Far below (y >
// 126) n is -126.
__device__ __forceinline__ uint64_t weigh(float z, float M, Two c, const Power* tab, int& k) {
  const Two d = two_sum(z, -M);
  const float p = __fmul_rn(d.h, c.h);
  const float pe = fmaf(d.h, c.h, -p) + fmaf(d.h, c.l, __fmul_rn(d.l, c.h));
  const float t = to_grid(p);
  k = steps_of(t);
  const float fh = __fsub_rn(p, __fsub_rn(t, kRound));  // exact
  const float f = __fadd_rn(fh, pe);
  constexpr float l1h = 0.6931471824645996f, l1l = -1.9046542e-09f;  // ln 2
  const float a = __fmul_rn(fh, l1h);
  float ae = fmaf(pe, l1h, fmaf(fh, l1l, fmaf(fh, l1h, -a)));
  ae = fmaf(__fmul_rn(f, f), fmaf(f, 0.05550411f, 0.2402265f), ae);  // ln2^3 / 6, ln2^2 / 2
  const Power w = tab[k & 255];
  const float v = __fmul_rn(w.h, a);
  const float ve = fmaf(w.l, a, fmaf(w.h, ae, fmaf(w.h, a, -v)));
  constexpr float kOne = (float)(1ull << kFrac);
  const int more = __float2int_rn(v * kOne) + __float2int_rn(ve * kOne);  // within 2^31
  return z == M ? 1ull << kFrac : w.whole + (long long)more;
}

// What all lanes hold anyway, told to the compiler: a branch on it then needs no
// reconvergence before each of the shuffles inside (the draw's sums and choice by one warp:
// 1450 cycles, 9100 without).
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(kAll, v, 0); }
__device__ __forceinline__ float uniform(float v) { return __shfl_sync(kAll, v, 0); }

// Tokens of a thread's run; odd, so that the threads of a warp read different banks.
template <int kC, int kT>
__host__ __device__ __forceinline__ int each_of(int V) {
  return ((V + kC * kT - 1) / (kC * kT)) | 1;
}

// held: the row's parts fit the blocks' shared memory; else they are read again from global.
template <int kC, int kT, bool held>
__global__ void __launch_bounds__(kT, 512 / kT) k_sample_filtered(FilteredArgs a, FastDiv by_each) {
  constexpr int kW = kT / 32, kN = kC * kW, kBins = kBinsOf<kC>;
  static_assert(kN <= 64, "two warps a lane");
  static_assert(kT >= 256, "a power of two of the table a thread");
  __shared__ Shared<kC, kW> sh;
  extern __shared__ __align__(16) unsigned char dyn[];
  unsigned long long* const columns = reinterpret_cast<unsigned long long*>(dyn);  // [kBins][kT]
  unsigned long long* const column = columns + threadIdx.x;
  float* const hold = reinterpret_cast<float*>(columns + kBins * kT);
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
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  // the other blocks' shared memory can be written once they have started
  if (tid == 0) sh.taken = 0;
  if constexpr (kC > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  if (tid < 256) {  // 2^(k/256) = 2^(k/8 / 32) 2^(k%8 / 256)
    constexpr float2 kFine[8] = {
        {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.00b1b00000000p+0f, -0x1.6950d00000000p-26f},
        {0x1.0163da0000000p+0f, 0x1.3f66660000000p-25f}, {0x1.0216820000000p+0f, -0x1.789fb00000000p-25f},
        {0x1.02c9a40000000p+0f, -0x1.887fa00000000p-28f}, {0x1.037d420000000p+0f, 0x1.c2377a0000000p-25f},
        {0x1.04315e0000000p+0f, 0x1.0dcff00000000p-25f}, {0x1.04e5f80000000p+0f, -0x1.a1356a0000000p-25f}};
    float2 fine = kFine[0];
#pragma unroll
    for (int i = 1; i < 8; ++i)
      if ((tid & 7) == i) fine = kFine[i];
    const float2 e = kExp2[tid >> 3];
    const Two w = mul({e.x, e.y}, {fine.x, fine.y});
    sh.tab[tid] = {(uint64_t)(w.h * (float)(1ull << kFrac)) + (long long)rintf(w.l * (float)(1ull << kFrac)), w.h, w.l};
  }
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x / kC, V = a.V;
  const float temp = uniform(a.temps[row]), u_row = a.u[row];
  const int top_k = uniform(a.top_k ? a.top_k[row] : 0);
  const float top_p = uniform(a.top_p ? a.top_p[row] : 1.0f), min_p = uniform(a.min_p ? a.min_p[row] : 0.0f);
  const int each = each_of<kC, kT>(V);
  const int base = (int)min((int64_t)V, (int64_t)rank * kT * each);
  const int count = (int)min((int64_t)V - base, (int64_t)kT * each);
  const int run = tid * each, hi = min(count, run + each);
  const float* const z_row = a.logits + row * a.ld + base;
  // ---- the row and its maximum
  float M = -CUDART_INF_F;
  // eight vectors asked for at once: the blocks of a wave start together, and wait for these
  // (256 rows of 49152 from HBM, top-p: 100 us, 114 with a bound to check between them)
  auto look = [&](auto n, auto one, int i0) {
    constexpr int kOne = decltype(one)::value;  // tokens of a load
    using Raw = std::conditional_t<kOne == 4, float4, float>;
    Raw v[n];
#pragma unroll
    for (int q = 0; q < n; ++q) v[q] = *reinterpret_cast<const Raw*>(z_row + i0 + q * kOne * kT);
#pragma unroll
    for (int q = 0; q < n; ++q) {
      if constexpr (kOne == 4) {
        v[q].x = clean(v[q].x), v[q].y = clean(v[q].y), v[q].z = clean(v[q].z), v[q].w = clean(v[q].w);
        M = fmaxf(M, fmaxf(fmaxf(v[q].x, v[q].y), fmaxf(v[q].z, v[q].w)));
      } else {
        v[q] = clean(v[q]);
        M = fmaxf(M, v[q]);
      }
      if (held) *reinterpret_cast<Raw*>(hold + i0 + q * kOne * kT) = v[q];
    }
  };
  auto look_from = [&](auto one, int from, int to) {  // to - from: whole loads
    constexpr int kOne = decltype(one)::value;
    int i = from + kOne * tid;
    for (; i + 7 * kOne * kT < to; i += 8 * kOne * kT) look(std::integral_constant<int, 8>{}, one, i);
    for (; i < to; i += kOne * kT) look(std::integral_constant<int, 1>{}, one, i);
  };
  const int vectors = (reinterpret_cast<uintptr_t>(z_row) & 15) == 0 ? count & ~3 : 0;
  look_from(std::integral_constant<int, 4>{}, 0, vectors);
  look_from(std::integral_constant<int, 1>{}, vectors, count);
  if (held)
    for (int i = count + tid; i < kT * each; i += kT) hold[i] = -CUDART_INF_F;
  M = warp_max(M);
#pragma unroll
  for (int b = 0; b < kBins; ++b) column[b * kT] = 0;
  if constexpr (kC > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (lane < kC) *remote(&sh.max[rank * kW + warp], lane) = M;
  // only the first in rank stays: of the largest logits the lowest index
  const bool only = !(temp > 0.0f) || min_p > 1.0f;
  const Two c = log2e_over(only ? 1.0f : fminf(fmaxf(temp, 1e-30f), 1e30f));
  sync();
  const int e0 = 2 * lane, e1 = 2 * lane + 1;  // a lane's warps of the cluster
  M = uniform(warp_max(fmaxf(e0 < kN ? sh.max[e0] : -CUDART_INF_F, e1 < kN ? sh.max[e1] : -CUDART_INF_F)));
  auto at = [&](int i) { return held ? hold[i] : i < count ? clean(z_row[i]) : -CUDART_INF_F; };
  if (only || M == -CUDART_INF_F) {
    int first = V;
    for (int i = tid; i < count; i += kT)
      if (at(i) == M && first == V) first = base + i;
    first = __reduce_min_sync(kAll, first);
    if (lane == 0) *remote(&sh.at[rank * kW + warp], 0) = first;
    sync();
    if (rank != 0 || warp != 0) return;
    first = __reduce_min_sync(kAll, min(e0 < kN ? sh.at[e0] : V, e1 < kN ? sh.at[e1] : V));
    if (lane == 0) {
      a.tokens[row] = M > -CUDART_INF_F ? first : 0;
      if (a.kept) a.kept[row] = M > -CUDART_INF_F ? 1 : 0;
    }
    return;
  }
  const bool by_k = top_k > 0 && top_k < V, by_p = top_p < 1.0f, by_m = min_p > 0.0f;
  // the bin, of those from y = from on: below 0 for what lies ahead of them
  auto bin_of = [](int k, int from) { return min(kBins - 1, -(k >> 8) - from); };
  // min-p ends in y's bins m_first to m_last (of kNone bins)
  constexpr int kNone = 1 << 20;
  int m_first = kNone, m_last = kNone;
  if (by_m) {
    const float y = fminf(-lg2(min_p), 200.0f);  // bin b has y from b - 1 to b, 1/512 less or more
    m_first = (int)floorf(y - 0.01f) + 1;
    m_last = (int)(y + 1.02f);
  }

  // The columns' bins are those from y = off on, of which a thread has ahead_sum (of 2^-54) and
  // ahead_n in front.
  int off = 0, ahead_n = 0;
  uint64_t ahead_sum = 0;
  // A weight as a whole number of 2^-(off + bin + kFrac): in the last bin what is left of it, and
  // 1 where nothing is, so that the first of them can be drawn (by u = 0). 2^20 such ones are
  // 2^-38 of the sum.
  auto mass_of = [&](float z, int from, int& bin) {
    int k;
    const uint64_t m = weigh(z, M, c, sh.tab, k);
    const int b = -(k >> 8) - from;
    bin = min(kBins - 1, b);
    const uint64_t left = m >> min(63, b - bin);
    return k > kLeast ? left | (left == 0) : 0;
  };
  auto mass = [&](float z) {
    int bin;
    return mass_of(z, off, bin);
  };
  auto weight = [&](float z) {  // times 2^60
    int k;
    const uint64_t m = weigh(z, M, c, sh.tab, k);
    return to_two(k > kLeast ? m : 0, (k >> 8) - kFrac + 60);
  };
  // ---- counts and masses of the bins
  // Four tokens in step, without branches, so that their chains of dependent operations
  // overlap; for -inf, which also stands behind the row's end, nothing is added.
  const bool few = by_k && top_k <= kFew;  // no weights are wanted
  auto count_bins = [&](auto weighed, auto all) {
    const int from = decltype(all)::value ? 0 : off;
    auto step = [&](auto n, int j) {
      int b[n];
      unsigned long long m[n];
#pragma unroll
      for (int q = 0; q < n; ++q) {
        const float z = at(run + j + q);
        if constexpr (decltype(weighed)::value) m[q] = mass_of(z, from, b[q]);
        else m[q] = 0, b[q] = bin_of(place(z, M, c), from);
        bool in = z > -CUDART_INF_F;
        if constexpr (!decltype(all)::value) in = in && b[q] >= 0, b[q] = max(b[q], 0);
        m[q] = in ? m[q] + (1ull << kCount) : 0;
      }
#pragma unroll
      for (int q = 0; q < n; ++q) column[b[q] * kT] += m[q];
    };
    int j = 0;
    for (; j + 4 <= each; j += 4) step(std::integral_constant<int, 4>{}, j);
    for (; j < each; ++j) step(std::integral_constant<int, 1>{}, j);
  };
  if (few) count_bins(std::false_type{}, std::true_type{});
  else count_bins(std::true_type{}, std::true_type{});
  // a thread's mass (of 2^-54) and count in bins up to `to`
  auto add_bins = [&](int to, uint64_t& sum, int& n) {
#pragma unroll
    for (int b = 0; b < kBins; ++b) {
      const uint64_t v = b <= to ? column[b * kT] : 0, m = v & ((1ull << kCount) - 1);
      n += (int)(v >> kCount);
      const int s = 54 - kFrac - b - off;
      sum += s >= 0 ? m << s : (m + (1ull << min(-s, 62)) - 1) >> min(-s, 62);  // rounded up: none is lost
    }
  };
  // The tokens of a bin, each warp's own; f(z, i) for each of them, every lane another.
  // Their places lie in the warp's columns of the bins behind, which no one wants any more,
  // 128 a bin; a warp that has more of them, or whose row is not held, looks at its runs.
  int members_of = -1, gathered_n = 0;
  bool in_columns = false;
  auto place_of = [&](int k) {
    return reinterpret_cast<uint16_t*>(columns + (members_of + 1 + (k >> 7)) * kT + warp * 32) + (k & 127);
  };
  auto gather = [&](int bin) {
    if (members_of == bin) return;
    members_of = bin;
    if (!held) return;
    __syncwarp();
    const int room = (kBins - 1 - bin) * 128;
    // the bin's places, on the grid: from the last token's to the first's
    const float t0 = bin < kBins - 1 ? kRound - (float)(off + bin) : 0.0f, t1 = kRound - (float)(off + bin) + 255.0f / 256.0f;
    int n = 0;
    for (int j0 = 0; j0 < each; j0 += 32) {  // 32 tokens of each lane: which, how many, where to
      unsigned in = 0;
      const int some = min(32, each - j0);
      auto look = [&](auto n, int j) {
        float z[n];
        unsigned m = 0;
#pragma unroll
        for (int q = 0; q < n; ++q) z[q] = hold[run + j0 + j + q];
#pragma unroll
        for (int q = 0; q < n; ++q) {
          const float t = to_grid(__fmul_rn(__fadd_rn(z[q], -M), c.h));
          if (t >= t0 && t <= t1 && z[q] > -CUDART_INF_F) m |= 1u << q;
        }
        in |= m << j;
      };
      int j = 0;
      for (; j + 8 <= some; j += 8) look(std::integral_constant<int, 8>{}, j);
      for (; j < some; ++j) look(std::integral_constant<int, 1>{}, j);
      int k = __popc(in), upto = k;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(kAll, upto, o);
        if (lane >= o) upto += up;
      }
      k = n + upto - k;
      n += __shfl_sync(kAll, upto, 31);
      for (; in; in &= in - 1, ++k)
        if (k < room) *place_of(k) = (uint16_t)(run + j0 + __ffs(in) - 1);
    }
    gathered_n = uniform(n);
    in_columns = gathered_n <= room;
    __syncwarp();
  };
  auto members = [&](auto f) {  // f(z[4], i[4], in[4])
    float z[4];
    int i[4];
    bool in[4];
    if (held && in_columns) {
      for (int j = lane; j < gathered_n; j += 128) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          in[q] = j + 32 * q < gathered_n;
          i[q] = *place_of(in[q] ? j + 32 * q : lane);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) z[q] = hold[i[q]];
        f(z, i, in);
      }
    } else {
      for (int j = run; j < hi; j += 4) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          i[q] = min(j + q, hi - 1);
          z[q] = at(i[q]);
          in[q] = j + q < hi && z[q] > -CUDART_INF_F && bin_of(place(z[q], M, c), off) == members_of;
        }
        f(z, i, in);
      }
    }
  };
  int cut_bin = kNone;               // of y's: all ahead of it stay whole
  uint64_t cut = ~0ull;              // the last rank that stays
  const Two least = {min_p * kUp, 0.0f};
  if (by_k || by_p) {
    auto exchange = [&] {  // the bins' counts and masses, to every block
      for (int b = warp; b < kBins; b += kW) {
        unsigned long long m = 0;
        uint32_t n = 0;
  #pragma unroll
        for (int j = 0; j < kT; j += 32) {
          const unsigned long long v = columns[b * kT + j + lane];
          n += (uint32_t)(v >> kCount);
          m += v & ((1ull << kCount) - 1);
        }
        constexpr uint32_t kLimb = (1u << 24) - 1;
        const unsigned long long sum = (unsigned long long)__reduce_add_sync(kAll, (uint32_t)m & kLimb) +
                                       ((unsigned long long)__reduce_add_sync(kAll, (uint32_t)(m >> 24) & kLimb) << 24) +
                                       ((unsigned long long)__reduce_add_sync(kAll, (uint32_t)(m >> 48)) << 48);
        n = __reduce_add_sync(kAll, n);
        if (lane < kC) *remote(&sh.bins[rank][b], lane) = Bin{sum, n, 0};
      }
      sync();
    };
    __syncthreads();
    exchange();
    // The columns with the bins from y = to on, 0 or a later one. The tokens of a cut far out
    // (the tail of a peaked row) are in the last bin, with most others, or have no room behind
    // theirs: another count takes less time than walks through all tokens (64 rows of 49152, T =
    // 0.6, top-p 0.998: 38 us, 127 by walks).
    auto move = [&](int to) {
      if (to == 0) ahead_sum = 0, ahead_n = 0;
      else add_bins(to - off - 1, ahead_sum, ahead_n);
      off = to;
      members_of = -1;
      __syncwarp();
#pragma unroll
      for (int b = 0; b < kBins; ++b) column[b * kT] = 0;
      if (few) count_bins(std::false_type{}, std::false_type{});
      else count_bins(std::true_type{}, std::false_type{});
      sync();  // also: the last bins have been read
      exchange();
    };
    // Looks for the first rank whose running count reaches `need` (by_count) or whose running
    // mass reaches `goal` (times 2^60). False: it is `cut`, and the running mass is `upto`.
    // True: it is among the first `upto_n` ranks, which are in block 0's list `which`.
    auto find = [&](bool by_count, uint32_t need, Two goal, int which, Two& upto, int& upto_n) {
      upto = {0.0f, 0.0f};
      uint32_t ahead = 0, left = 0;
      Two before = {0.0f, 0.0f};
      // of parts' counts and masses (of `n` parts, the blocks' `apart`), the one with the
      // target: by the first warp, for all
      auto choose = [&](const Bin* parts, int apart, int parts_n, int unit) {
        if (warp == 0) {
          uint32_t n[2] = {0, 0};
          Two m[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int i = 2 * lane + q;
            uint64_t sum = 0;
            if (i < parts_n)
#pragma unroll
              for (int r = 0; r < kC; ++r) n[q] += parts[r * apart + i].count, sum += parts[r * apart + i].mass;
            m[q] = to_two(sum, 60 - kFrac - off - (unit < 0 ? min(i, kBins - 1) : unit));
          }
          uint32_t n_in = n[0] + n[1];
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(kAll, n_in, o);
            if (lane >= o) n_in += up;
          }
          const Two m_in = add(before, scan(add(m[0], m[1]), lane));
          const bool reach = by_count ? ahead + n_in >= need : !less(m_in, goal);
          const unsigned has = __ballot_sync(kAll, n[0] + n[1] > 0);
          const unsigned hit = __ballot_sync(kAll, n[0] + n[1] > 0 && reach);
          const int p = hit ? __ffs(hit) - 1 : 31 - __clz(has);
          if (p > 0) {
            before = shfl(m_in, p - 1);
            ahead += __shfl_sync(kAll, n_in, p - 1);
          }
          const uint32_t n0 = __shfl_sync(kAll, n[0], p), n1 = __shfl_sync(kAll, n[1], p);
          const Two half = add(before, shfl(m[0], p));
          const bool first = n0 > 0 && (n1 == 0 || (hit && (by_count ? ahead + n0 >= need : !less(half, goal))));
          if (!first) before = half, ahead += n0;
          if (lane == 0) sh.found = {before, ahead, first ? n0 : n1, 2 * p + !first};
        }
        __syncthreads();
        before = sh.found.before;
        ahead = (uint32_t)uniform((int)sh.found.ahead), left = (uint32_t)uniform((int)sh.found.left);
        return uniform(sh.found.at);
      };
      // a list, and top-p's sum, want the cut wherever it is, and no columns
      const bool cut_only = few || (by_count && by_p);
      int bin, next = off ? 0 : -1;  // top-k's cut was far out
      for (;;) {
        if (next >= 0) move(next);
        bin = choose(&sh.bins[0][0], kBins, kBins, -1);
        if (!cut_only && m_last < off + bin) return false;  // min-p ends ahead of it
        // 7/8 of the warps' room for them
        const bool fits = held ? left <= (uint32_t)((kBins - 1 - bin) * 112 * kN) : bin < kBins - 1;
        if (fits || bin == 0 || off + bin > 126 || (!cut_only && m_first < off + bin)) break;
        next = off + bin;
      }
      int part = -1;
      uint64_t from = 0, to = ~0ull;
      auto each_left = [&](auto f) {  // f(z[4], rank[4], in[4])
        gather(bin);
        members([&](const float (&z)[4], const int (&i)[4], bool (&in)[4]) {
          uint64_t r[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            r[q] = rank_of(z[q], base + i[q]);
            in[q] = in[q] && (part < 0 || part_of(place(z[q], M, c), off + bin) == part) && from <= r[q] && r[q] <= to;
          }
          f(z, r, in);
        });
      };
      const Bin* from_blocks = &sh.bins[0][bin];  // the chosen part's entry of block 0, the blocks' apart
      int apart = kBins;
      bool ranged = false;
      for (int level = 0; left > kList || (by_count && need <= kFew && ahead + left > kList); ++level) {
        const bool by_y = bin < kBins - 1 && part < 0;
        if (!by_y && !ranged) {  // the members' first and last rank
          if (tid == 0) sh.lo = ~0ull, sh.hi = 0;
          __syncthreads();
          unsigned long long l = ~0ull, h = 0;
          each_left([&](const float (&)[4], const uint64_t (&r)[4], const bool (&in)[4]) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (in[q]) l = min(l, (unsigned long long)r[q]), h = max(h, (unsigned long long)r[q]);
          });
          if (l <= h) atomicMin(&sh.lo, l), atomicMax(&sh.hi, h);
          __syncthreads();
          if (tid < kC) {
            uint64_t* const to_block = remote(&sh.range[rank][0], tid);
            to_block[0] = sh.lo, to_block[1] = sh.hi;
          }
          sync();
          from = ~0ull, to = 0;
          for (int r = 0; r < kC; ++r) {
            from = min(from, sh.range[r][0]);
            to = max(to, sh.range[r][1]);
          }
          ranged = true;
        }
        const int shift = max(0, 64 - __clzll((long long)(to - from)) - 6);
        for (int t = tid; t < 4 * kSub; t += kT) sh.own[t / kSub][t % kSub] = 0;
        if (level) sync();  // the last level's parts have been read
        else __syncthreads();
        // a mass in three parts of 13 and 14 bits: 2^17 of them fit 32 bits
        each_left([&](const float (&z)[4], const uint64_t (&r)[4], const bool (&in)[4]) {
          uint64_t m[4] = {};
          if (!few)
#pragma unroll
            for (int q = 0; q < 4; ++q) m[q] = mass(z[q]);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (in[q]) {
              const int p = by_y ? part_of(place(z[q], M, c), off + bin) : (int)((r[q] - from) >> shift);
              if (!few) {
                atomicAdd(&sh.own[0][p], (uint32_t)m[q] & 0x1fff);
                atomicAdd(&sh.own[1][p], (uint32_t)(m[q] >> 13) & 0x1fff);
                atomicAdd(&sh.own[2][p], (uint32_t)(m[q] >> 26));
              }
              atomicAdd(&sh.own[3][p], 1u);
            }
        });
        __syncthreads();
        for (int t = tid; t < kC * kSub; t += kT) {
          const int p = t % kSub;
          const uint64_t m = sh.own[0][p] + ((uint64_t)sh.own[1][p] << 13) + ((uint64_t)sh.own[2][p] << 26);
          *remote(&sh.sub[rank][p], t / kSub) = Bin{m, sh.own[3][p], 0};
        }
        sync();
        const int p = choose(&sh.sub[0][0], kSub, kSub, bin);
        if (by_y) {
          part = p;
        } else {
          from += (uint64_t)p << shift;
          to = min(to, from + ((uint64_t)1 << shift) - 1);
        }
        from_blocks = &sh.sub[0][p];
        apart = kSub;
      }
      if (ahead + left <= kList) {  // all ranks up to the part's last, to block 0
        for (int i = run; i < hi; ++i) {
          const float z = at(i);
          const int k = place(z, M, c), b = bin_of(k, off);
          if (!(z > -CUDART_INF_F) || b > bin) continue;
          const uint64_t r = rank_of(z, base + i);
          if (b == bin && ((part >= 0 && part_of(k, off + bin) > part) || r > to)) continue;
          *remote(&sh.list[which][atomicAdd(remote(&sh.taken, 0), 1)], 0) = r;
        }
        upto_n = (int)(ahead + left);
        sync();
        return true;
      }
      // the members, to every block
      int place = 0;
      for (int r = 0; r < rank; ++r) place += from_blocks[r * apart].count;
      if (tid == 0) sh.fill = place, sh.hit = kList;
      __syncthreads();
      each_left([&](const float (&)[4], const uint64_t (&r)[4], const bool (&in)[4]) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (in[q]) {
            const int p = atomicAdd(&sh.fill, 1);
#pragma unroll
            for (int b = 0; b < kC; ++b) *remote(&sh.list[which][p], b) = r[q];
          }
      });
      sync();
      const int n = (int)left;
      static_assert(kList <= kT, "a thread a token");
      if (tid < n) {
        const uint64_t mine = sh.list[which][tid];
        int p = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) p += sh.list[which][j] < mine;
        sh.sorted[p] = mine;
      }
      __syncthreads();
      if (warp < kList / 32) {
        Two in = scan(tid < n ? weight(logit_of(sh.sorted[tid])) : Two{0.0f, 0.0f}, lane);
        if (lane == 31) sh.scan[warp] = in;
        asm volatile("bar.sync 1, %0;" ::"n"(kList) : "memory");
        for (int w = 0; w < warp; ++w) before = add(before, sh.scan[w]);
        in = add(before, in);
        if (tid < n && (by_count ? tid + 1 + ahead == need : !less(in, goal))) atomicMin(&sh.hit, tid);
        asm volatile("bar.sync 1, %0;" ::"n"(kList) : "memory");
        if (tid == min(sh.hit, n - 1)) sh.scan[kW - 1] = in;
      }
      static_assert(kW > kList / 32, "a place of the sums' for the answer");
      __syncthreads();
      upto = sh.scan[kW - 1];
      cut_bin = min(cut_bin, off + bin);
      cut = min(cut, sh.sorted[uniform(min(sh.hit, n - 1))]);
      return false;
    };
    Two sum = {0.0f, 0.0f};
    if (!by_k) {
      uint64_t m = 0;
      if (lane < kBins)
        for (int r = 0; r < kC; ++r) m += sh.bins[r][lane].mass;
      sum = to_two(m, 60 - kFrac - min(lane, kBins - 1));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum = add(sum, shfl_xor(sum, o));
    }
    int first_n = 0, which = 0;
    bool listed = false, k_in = false;  // the first ranks are in a list; top-k's end too
#pragma unroll 1  // one copy of the search
    for (int p = by_k ? 0 : 1; p < (by_p ? 2 : 1) && !listed; ++p) {
      if (p) __syncthreads();  // sh.hit and sh.scan have been read
      which = p;
      Two upto;
      listed = find(!p, (uint32_t)top_k, mul({fmaxf(top_p, 0.0f), 0.0f}, sum), p, upto, first_n);
      if (!p) sum = upto, k_in = listed;
    }
    if (listed) {
      // ---- everything else in one block: a thread a rank, then a thread an index
      if (rank != 0 || warp >= kList / 32) return;
      auto meet = [] { asm volatile("bar.sync 1, %0;" ::"n"(kList) : "memory"); };
      const int n = first_n;
      if (tid < n) {
        const uint64_t mine = sh.list[which][tid];
        int p = 0;
#pragma unroll 4
        for (int j = 0; j < n; ++j) p += sh.list[which][j] < mine;
        sh.sorted[p] = mine;
      }
      if (tid == 0) sh.hit = kList, sh.fill = 0;
      meet();
      // running sums over the 128 threads
      auto run_sum = [&](Two v) {
        Two in = scan(v, lane);
        meet();  // the last sums have been read
        if (lane == 31) sh.scan[warp] = in;
        meet();
        Two ahead = {0.0f, 0.0f};
        for (int w = 0; w < warp; ++w) ahead = add(ahead, sh.scan[w]);
        return add(ahead, in);
      };
      const uint64_t mine = tid < n ? sh.sorted[tid] : ~0ull;
      const Two w = tid < n ? weight(logit_of(mine)) : Two{0.0f, 0.0f};
      int stay = k_in ? min(n, top_k) : n;
      if (by_p) {
        const Two in = run_sum(tid < stay ? w : Two{0.0f, 0.0f});
        if (k_in) {
          if (tid == stay - 1) sh.found.before = in;
          meet();
          sum = sh.found.before;
        }
        if (tid < stay && !less(in, mul({fmaxf(top_p, 0.0f), 0.0f}, sum))) atomicMin(&sh.hit, tid);
        meet();
        stay = min(stay, sh.hit + 1);
      }
      const bool kept = tid < stay && (!by_m || !less(w, least));
      if (kept) {
        atomicAdd(&sh.fill, 1);
      }
      meet();
      stay = sh.fill;  // a prefix: weights fall with the rank
      if (tid == 0 && a.kept) a.kept[row] = stay;
      // by index
      if (tid < stay) {
        int p = 0;
#pragma unroll 4
        for (int j = 0; j < stay; ++j) p += (uint32_t)sh.sorted[j] < (uint32_t)mine;
        sh.list[which][p] = mine;
      }
      if (tid == 0) sh.hit = kList;
      meet();
      const uint64_t token = tid < stay ? sh.list[which][tid] : 0;
      const Two v = tid < stay ? weight(logit_of(token)) : Two{0.0f, 0.0f};
      const Two in = run_sum(v);
      if (tid == stay - 1) sh.found.before = in;
      meet();
      if (v.h > 0.0f && !less(in, mul({fminf(u_row, 1.0f), 0.0f}, sh.found.before))) atomicMin(&sh.hit, tid);
      if (tid == 0) sh.fill = -1;
      meet();
      if (v.h > 0.0f) atomicMax(&sh.fill, tid);
      meet();
      if (tid == 0) a.tokens[row] = (int)(uint32_t)sh.list[which][sh.hit < kList ? sh.hit : sh.fill];
      return;
    }
  }
  // ---- bins that stay whole, and those that are looked at token by token: the cut's, and
  // the one or two where min-p may end
  int whole = min(cut_bin, m_first) - off;
  if (by_m || cut_bin < kNone) whole = max(0, min(whole, kBins - 1));
  const int last = min(min(cut_bin, m_last) - off, kBins - 1);
  auto stays = [&](float z, int i) { return rank_of(z, base + i) <= cut && (!by_m || !less(weight(z), least)); };
  for (int b = whole; b <= last; ++b) {
    gather(b);
    __syncwarp();
    column[b * kT] = 0;
    __syncwarp();
    members([&](const float (&z)[4], const int (&i)[4], const bool (&in)[4]) {
      uint64_t m[4];
      bool stay[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) m[q] = mass(z[q]), stay[q] = stays(z[q], i[q]);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (in[q] && stay[q]) atomicAdd(columns + b * kT + by_each.div((uint32_t)i[q]), m[q] + (1ull << kCount));
    });
  }
  __syncwarp();
  // ---- kept mass and count of the runs
  Kept mine = {{0.0f, 0.0f}, 0};
  {
    uint64_t sum = ahead_sum;
    mine.count = ahead_n;
    add_bins(last, sum, mine.count);
    mine.mass = to_two(sum, 60 - 54);
  }
  const Two in = scan(mine.mass, lane);
  {
    const int n = __reduce_add_sync(kAll, mine.count);
    const Two m = shfl(in, 31);
    if (lane < kC) *remote(&sh.kept[rank * kW + warp], lane) = Kept{m, n};
  }
  sync();
  // ---- the draw: the warp (found by one of each block), the lane, the token
  if (warp == 0) {
    const Kept none = {{0.0f, 0.0f}, 0};
    const Kept k0 = e0 < kN ? sh.kept[e0] : none, k1 = e1 < kN ? sh.kept[e1] : none;
    const int n = __reduce_add_sync(kAll, k0.count + k1.count);
    if (rank == 0 && lane == 0 && a.kept) a.kept[row] = n;
    Two total = add(k0.mass, k1.mass);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total = add(total, shfl_xor(total, o));
    const Two goal = mul({fminf(u_row, 1.0f), 0.0f}, total);
    Two cum = {0.0f, 0.0f};
    const int chosen = pick(k0.mass, k1.mass, goal, cum, lane);
    if (lane == 0) sh.found.before = cum, sh.found.at = chosen, sh.scan[0] = goal;
  }
  __syncthreads();
  Two cum = sh.found.before;
  const Two goal = sh.scan[0];
  if (uniform(sh.found.at) != rank * kW + warp) return;
  const unsigned reach = __ballot_sync(kAll, mine.mass.h > 0.0f && !less(add(cum, in), goal));
  const unsigned has = __ballot_sync(kAll, mine.mass.h > 0.0f);
  const int who = reach ? __ffs(reach) - 1 : 31 - __clz(has);
  if (who > 0) cum = add(cum, shfl(in, who - 1));
  const int start = __shfl_sync(kAll, run, who), end = __shfl_sync(kAll, hi, who);
  int found = -1, last_in = -1;
  for (int i0 = start; i0 < end && found < 0; i0 += 32) {
    const int i = i0 + lane;
    Two w = {0.0f, 0.0f};
    if (i < end) {
      const float z = at(i);
      if (z > -CUDART_INF_F && stays(z, i)) w = weight(z);
    }
    const Two s = add(cum, scan(w, lane));
    const unsigned h = __ballot_sync(kAll, w.h > 0.0f);
    const unsigned r = __ballot_sync(kAll, w.h > 0.0f && !less(s, goal));
    cum = shfl(s, 31);
    if (r) found = i0 + __ffs(r) - 1;
    if (h) last_in = i0 + 31 - __clz(h);
  }
  if (lane == 0) a.tokens[row] = base + (found >= 0 ? found : last_in);
}

// Bytes of dynamic shared memory that a block can have.
template <int kC, int kT>
constexpr int kRoom = 227 * 1024 - (int)((sizeof(Shared<kC, kT / 32>) + 1023) / 1024 * 1024);

template <int kC, int kT, bool kHeld>
Launched launch_h(const FilteredArgs& a, cudaStream_t s) {
  auto kernel = k_sample_filtered<kC, kT, kHeld>;
  static std::atomic<uint64_t> done{0};
  Launched l;
  l.error = allow_smem(kernel, kRoom<kC, kT>, done);
  if (l.error != cudaSuccess) return l;
  const int each = each_of<kC, kT>(a.V);
  const int64_t smem = (int64_t)kBinsOf<kC> * kT * 8 + (kHeld ? kT * (int64_t)each * 4 : 0);
  const FastDiv by_each((uint32_t)each);
  if constexpr (kC == 1) l.add(launch_k(kernel, dim3((unsigned)a.n), kT, smem, s, a, by_each));
  else l.add(launch_k_cluster(kernel, dim3((unsigned)a.n * kC), kT, smem, s, kC, a, by_each));
  return l;
}

// About how long a call takes (us), or infinity where a row's parts do not fit the blocks' shared
// memory or their places 16 bits.
template <int kC, int kT>
double estimate(const FilteredArgs& a, int sms) {
  const int64_t mine = kT * (int64_t)each_of<kC, kT>(a.V), smem = (int64_t)kBinsOf<kC> * kT * 8 + mine * 4;
  if (smem > kRoom<kC, kT> || mine > 65536) return HUGE_VAL;
  // blocks an SM; clusters of four and eight leave some of a GPC's SMs over
  const int two = kT == 256 && smem <= kRoom<kC, kT> - 114 * 1024 ? 2 : 1;
  const int usable = kC == 8 ? sms * 3 / 4 : kC == 4 ? sms * 7 / 8 : sms;
  const int at_once = std::max(1, usable * two / kC);
  const double row = 8.5 + (kC == 8 ? 2.4 : kC == 4 ? 1.6 : kC == 2 ? 0.8 : 0.0) + (kT == 512 ? 1.5 : 0.0) +
                     (kT == 512 ? 0.56e-3 : 0.74e-3) * a.V / kC;
  return (double)((a.n + at_once - 1) / at_once) * row * ((int64_t)a.n * kC > usable ? 1.25 : 1.0);
}

}  // namespace

// More blocks a row make a row faster, and fewer rows at a time: the estimate of waves of rows
// decides. Measured, us, top-p 0.95, by a block of 256 threads | a block of 512 | two of 512 |
// four of 512 | eight of 256 (-: does not fit); what is taken in brackets:
//   vocab   rows: 1                           64                          256
//   2048    (8.4) | 8.3 | 8.2 | 7.5 | 7.2     (11) | 12 | 13 | 21 | 24    (12) | 20 | 39 | 62 | 66
//   8192    14 | 13 | 11 | 10 | (9.4)         16 | 16 | (16) | 29 | 31    (19) | 30 | 55 | 96 | 106
//   32000   29 | 28 | 21 | 18 | (17)          29 | 27 | (22) | 35 | 40    57 | (54) | 83 | 130 | 144
//   49152   - | - | 25 | 20 | (18)            - | - | (26) | 39 | 44      - | - | (98) | 147 | 157
//   131072  - | - | - | 29 | (23)             - | - | - | (58) | 110      - | - | - | (245) | 416
// (16 rows of 131072: 30 by four blocks, 45 by eight.) A vocabulary that no variant holds is
// read again from global memory for each pass.
Launched launch_sample_filtered(const FilteredArgs& a, int sms, cudaStream_t s) {
  double least = HUGE_VAL;
  Launched (*launch)(const FilteredArgs&, cudaStream_t) = launch_h<8, 256, false>;
  auto offer = [&](double us, Launched (*f)(const FilteredArgs&, cudaStream_t)) {
    if (us < least) least = us, launch = f;
  };
  offer(estimate<1, 256>(a, sms), launch_h<1, 256, true>);
  offer(estimate<1, 512>(a, sms), launch_h<1, 512, true>);
  offer(estimate<2, 512>(a, sms), launch_h<2, 512, true>);
  offer(estimate<4, 512>(a, sms), launch_h<4, 512, true>);
  offer(estimate<8, 256>(a, sms), launch_h<8, 256, true>);
  return launch(a, s);
}

}  // namespace fsk
