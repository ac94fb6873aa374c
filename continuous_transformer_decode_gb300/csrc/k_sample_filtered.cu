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
// 1e-6 of the sum): weights are good to 2^-36 (draw.cuh) and are summed as whole numbers
// of 2^-40 of their bin's largest weight, so that sums do not depend on their order; sums
// of bins, and a draw's running sums, are pairs of f32 numbers.
//
// One thread-block cluster serves a row and reads it once, into shared memory. A thread has
// a run of consecutive tokens and a column of the bins' counts and masses for itself (no
// atomics). What the draw needs, the kept mass of each run in order, is then the sum of a
// column's bins ahead of the cut; only the tokens of the cut's own bin are weighed again.

#include <cooperative_groups.h>

#include "draw.cuh"
#include "fs_internal.h"

namespace fsk {
namespace {

using namespace draw;

namespace cg = cooperative_groups;

constexpr int kBins = 24;   // of y: [b, b + 1), the last one also all above
constexpr int kSub = 32;    // parts of a bin that is split
constexpr int kList = 256;  // tokens that are ranked among themselves
constexpr int kFrac = 40;   // a mass in bin b is a whole number of 2^-(b + kFrac)
constexpr int kCount = 50;  // a column's entry: count << kCount | mass

struct Bin {
  uint64_t mass;
  uint32_t count, pad;
};
struct Best {
  float max;
  int at, tokens;
};
struct Kept {
  Two mass;
  int count;
};

template <int kC, int kW>
struct Shared {
  float2 tab[32];
  Best best[kC * kW];
  Kept kept[kC * kW];
  Bin bins[kC][kBins];
  Bin sub[2][kC][kSub];
  unsigned long long sub_mass[kSub];
  uint32_t sub_count[kSub];
  uint64_t range[2][kC][2];
  unsigned long long lo, hi;
  uint64_t list[2][kList], sorted[kList];
  Two scan[kW];
  int hit, fill;
};

__device__ __forceinline__ Two to_two(uint64_t m, int e) {  // m * 2^e
  const float h = __ull2float_rn(m);
  const float l = (float)(long long)(m - (uint64_t)h);
  const float s = __int_as_float((127 + e) << 23);
  return {h * s, l * s};
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
__device__ __forceinline__ float clean(float z) { return z == z ? z + 0.0f : -CUDART_INF_F; }

template <int kC, int kT>
__global__ void __launch_bounds__(kT) k_sample_filtered(FilteredArgs a, int held) {
  constexpr int kW = kT / 32, kN = kC * kW;
  static_assert(kN <= 64, "two warps a lane");
  __shared__ Shared<kC, kW> sh;
  extern __shared__ __align__(16) unsigned char dyn[];
  uint64_t* const column = reinterpret_cast<uint64_t*>(dyn) + threadIdx.x;  // [kBins] kT apart
  float* const hold = reinterpret_cast<float*>(dyn + (size_t)kBins * kT * 8);
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
  // the other blocks' shared memory can be written once they have started
  if constexpr (kC > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x / kC, V = a.V;
  const float temp = a.temps[row];
  const float us = fminf(a.u[row], 1.0f);
  const bool greedy = !(temp > 0.0f);
  const Two c = log2e_over(greedy ? 1.0f : fminf(fmaxf(temp, 1e-30f), 1e30f));
  // a thread's run; odd, so that the threads of a warp read different banks
  const int each = ((V + kC * kT - 1) / (kC * kT)) | 1;
  const int base = (int)min((int64_t)V, (int64_t)rank * kT * each);
  const int count = (int)min((int64_t)V - base, (int64_t)kT * each);
  const int lo = min(count, tid * each), hi = min(count, lo + each);
  const float* const z_row = a.logits + row * a.ld + base;
  // ---- the row, its maximum (lowest index) and how many tokens it has
  Best best = {-CUDART_INF_F, V, 0};
  auto take = [&](float z, int i) {
    best.tokens += z > -CUDART_INF_F;
    if (z > best.max) best.max = z, best.at = base + i;
  };
  if ((reinterpret_cast<uintptr_t>(z_row) & 15) == 0) {
#pragma unroll 4
    for (int i = 4 * tid; i < count; i += 4 * kT) {
      float4 v = load4(z_row, i, count, true);
      v.x = clean(v.x), v.y = clean(v.y), v.z = clean(v.z), v.w = clean(v.w);
      if (held) {
        if (i + 4 <= count) *reinterpret_cast<float4*>(hold + i) = v;
        else {
          hold[i] = v.x;
          if (i + 1 < count) hold[i + 1] = v.y;
          if (i + 2 < count) hold[i + 2] = v.z;
        }
      }
      take(v.x, i), take(v.y, i + 1), take(v.z, i + 2), take(v.w, i + 3);
    }
  } else {
#pragma unroll 4
    for (int i = tid; i < count; i += kT) {
      const float z = clean(z_row[i]);
      if (held) hold[i] = z;
      take(z, i);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m = __shfl_xor_sync(kAll, best.max, o);
    const int at = __shfl_xor_sync(kAll, best.at, o);
    if (m > best.max || (m == best.max && at < best.at)) best.max = m, best.at = at;
    best.tokens += __shfl_xor_sync(kAll, best.tokens, o);
  }
  if constexpr (kC > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (lane < kC) *remote(&sh.best[rank * kW + warp], lane) = best;
  sync();
  const int e0 = 2 * lane, e1 = 2 * lane + 1;  // a lane's warps of the cluster
  {
    const Best none = {-CUDART_INF_F, V, 0};
    const Best b0 = e0 < kN ? sh.best[e0] : none, b1 = e1 < kN ? sh.best[e1] : none;
    best = b0;
    if (b1.max > best.max || (b1.max == best.max && b1.at < best.at)) best.max = b1.max, best.at = b1.at;
    best.tokens += b1.tokens;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m = __shfl_xor_sync(kAll, best.max, o);
      const int at = __shfl_xor_sync(kAll, best.at, o);
      if (m > best.max || (m == best.max && at < best.at)) best.max = m, best.at = at;
      best.tokens += __shfl_xor_sync(kAll, best.tokens, o);
    }
  }
  const float M = best.max;
  if (greedy || best.tokens == 0) {
    if (rank == 0 && tid == 0) {
      a.tokens[row] = best.tokens ? best.at : 0;
      if (a.kept) a.kept[row] = best.tokens ? 1 : 0;
    }
    return;
  }
  const int top_k = a.top_k ? a.top_k[row] : 0;
  const float top_p = a.top_p ? a.top_p[row] : 1.0f, min_p = a.min_p ? a.min_p[row] : 0.0f;
  const bool by_k = top_k > 0 && top_k < best.tokens, by_p = top_p < 1.0f, by_m = min_p > 0.0f;

  auto at = [&](int i) { return held ? hold[i] : clean(z_row[i]); };
  auto y_of = [&](float z) { return z == M ? 0.0f : (M - z) * c.h; };
  auto bin_of = [&](float y) { return min(kBins - 1, (int)y); };
  auto mass_of = [&](float z, int b) {  // the weight as a whole number of 2^-(b + kFrac)
    const Two w = weight2(z, M, c, sh.tab);  // times 2^60
    const float s = __int_as_float((127 + b - 60 + kFrac / 2) << 23);
    const float h = w.h * s, t = rintf(h);
    return (int64_t)(int)t * (1 << (kFrac / 2)) +
           (int)rintf(((h - t) + w.l * s) * (float)(1 << (kFrac / 2)));
  };
  // ---- counts and masses of the bins
#pragma unroll
  for (int b = 0; b < kBins; ++b) column[b * kT] = 0;
#pragma unroll 2
  for (int i = lo; i < hi; ++i) {
    const float z = at(i);
    if (z > -CUDART_INF_F) {
      const int b = bin_of(y_of(z));
      column[b * kT] += (uint64_t)mass_of(z, b) + (1ull << kCount);
    }
  }
  int cut_bin = kBins;               // all bins ahead of it stay whole
  uint64_t cut = ~0ull;              // the last rank that stays
  if (by_k || by_p) {
    __syncthreads();
    for (int b = warp; b < kBins; b += kW) {
      uint64_t m = 0;
      uint32_t n = 0;
      const uint64_t* e = reinterpret_cast<const uint64_t*>(dyn) + b * kT;
      for (int j = lane; j < kT; j += 32) {
        const uint64_t v = e[j];
        n += (uint32_t)(v >> kCount);
        m += v & ((1ull << kCount) - 1);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m += __shfl_xor_sync(kAll, m, o);
      n = __reduce_add_sync(kAll, n);
      if (lane < kC) *remote(&sh.bins[rank][b], lane) = Bin{m, n, 0};
    }
    sync();
    int turn = 0;
    // The first rank whose running count reaches `need` (by_count) or whose running mass
    // reaches `goal`; that running mass goes to `upto`.
    auto find = [&](bool by_count, uint32_t need, Two goal, int which, Two& upto) -> uint64_t {
      Two before = {0.0f, 0.0f};
      uint32_t ahead = 0, members = 0;
      // of the parts' counts and masses (lane's part over all blocks), the one with the target
      auto choose = [&](uint32_t n, Two m) {
        uint32_t n_in = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t up = __shfl_up_sync(kAll, n_in, o);
          if (lane >= o) n_in += up;
        }
        const Two m_in = scan(m, lane);
        const bool reach = by_count ? ahead + n_in >= need : !less(add(before, m_in), goal);
        const unsigned has = __ballot_sync(kAll, n > 0);
        const unsigned hit = __ballot_sync(kAll, n > 0 && reach);
        const int p = hit ? __ffs(hit) - 1 : 31 - __clz(has);
        members = __shfl_sync(kAll, n, p);
        if (p > 0) {
          before = add(before, shfl(m_in, p - 1));
          ahead += __shfl_sync(kAll, n_in, p - 1);
        }
        return p;
      };
      uint32_t n = 0;
      uint64_t m = 0;
      if (lane < kBins)
        for (int r = 0; r < kC; ++r) n += sh.bins[r][lane].count, m += sh.bins[r][lane].mass;
      const int bin = choose(n, to_two(m, -kFrac - min(lane, kBins - 1)));
      int part = -1;
      uint64_t from = 0, to = ~0ull;
      auto part_of = [&](float y) { return min(kSub - 1, (int)((y - (float)bin) * (float)kSub)); };
      auto member = [&](float z, int i, float& y) {
        if (!(z > -CUDART_INF_F)) return false;
        y = y_of(z);
        if (bin_of(y) != bin || (part >= 0 && part_of(y) != part)) return false;
        const uint64_t r = rank_of(z, base + i);
        return from <= r && r <= to;
      };
      const Bin* from_blocks = nullptr;  // the chosen part's entry of block 0, the blocks' apart
      int apart = kBins;
      from_blocks = &sh.bins[0][bin];
      bool ranged = false;
      while (members > kList) {
        const bool by_y = bin < kBins - 1 && part < 0;
        if (!by_y && !ranged) {  // the members' first and last rank
          if (tid == 0) sh.lo = ~0ull, sh.hi = 0;
          __syncthreads();
          uint64_t l = ~0ull, h = 0;
          for (int i = lo; i < hi; ++i) {
            const float z = at(i);
            float y;
            if (member(z, i, y)) {
              const uint64_t r = rank_of(z, base + i);
              l = min(l, r), h = max(h, r);
            }
          }
          if (l <= h) atomicMin(&sh.lo, l), atomicMax(&sh.hi, h);
          __syncthreads();
          if (tid < kC) {
            remote(&sh.range[turn][rank][0], tid)[0] = sh.lo;
            remote(&sh.range[turn][rank][0], tid)[1] = sh.hi;
          }
          sync();
          from = ~0ull, to = 0;
          for (int r = 0; r < kC; ++r) {
            from = min(from, sh.range[turn][r][0]);
            to = max(to, sh.range[turn][r][1]);
          }
          turn ^= 1;
          ranged = true;
        }
        const int shift = max(0, 64 - __clzll((long long)(to - from)) - 5);
        if (tid < kSub) sh.sub_mass[tid] = 0, sh.sub_count[tid] = 0;
        __syncthreads();
        for (int i = lo; i < hi; ++i) {
          const float z = at(i);
          float y;
          if (member(z, i, y)) {
            const int p = by_y ? part_of(y) : (int)((rank_of(z, base + i) - from) >> shift);
            atomicAdd(&sh.sub_mass[p], (unsigned long long)mass_of(z, bin));
            atomicAdd(&sh.sub_count[p], 1u);
          }
        }
        __syncthreads();
        for (int t = tid; t < kC * kSub; t += kT)
          *remote(&sh.sub[turn][rank][t % kSub], t / kSub) = Bin{sh.sub_mass[t % kSub], sh.sub_count[t % kSub], 0};
        sync();
        n = 0, m = 0;
        for (int r = 0; r < kC; ++r) n += sh.sub[turn][r][lane].count, m += sh.sub[turn][r][lane].mass;
        const int p = choose(n, to_two(m, -kFrac - bin));
        if (by_y) {
          part = p;
        } else {
          from += (uint64_t)p << shift;
          to = min(to, from + ((uint64_t)1 << shift) - 1);
        }
        from_blocks = &sh.sub[turn][0][p];
        apart = kSub;
        turn ^= 1;
      }
      // the members, to every block
      int place = 0;
      for (int r = 0; r < rank; ++r) place += from_blocks[r * apart].count;
      if (tid == 0) sh.fill = place, sh.hit = kList;
      __syncthreads();
      for (int i = lo; i < hi; ++i) {
        const float z = at(i);
        float y;
        if (member(z, i, y)) {
          const int p = atomicAdd(&sh.fill, 1);
          for (int r = 0; r < kC; ++r) *remote(&sh.list[which][p], r) = rank_of(z, base + i);
        }
      }
      sync();
      const int m_n = (int)members;
      for (int t = tid; t < m_n; t += kT) {
        const uint64_t mine = sh.list[which][t];
        int p = 0;
        for (int j = 0; j < m_n; ++j) p += sh.list[which][j] < mine;
        sh.sorted[p] = mine;
      }
      __syncthreads();
      static_assert(kList <= kT, "a thread a token");
      Two w = {0.0f, 0.0f};
      if (tid < m_n) {
        w = weight2(logit_of(sh.sorted[tid]), M, c, sh.tab);
        w = {w.h * (1.0f / kUp), w.l * (1.0f / kUp)};
      }
      Two in = scan(w, lane);
      if (lane == 31) sh.scan[warp] = in;
      __syncthreads();
      const Two warps = scan(lane < kW ? sh.scan[lane] : Two{0.0f, 0.0f}, lane);
      if (warp) in = add(shfl(warps, warp - 1), in);
      in = add(before, in);
      if (by_count ? tid + 1 + ahead == need : tid < m_n && !less(in, goal)) atomicMin(&sh.hit, tid);
      __syncthreads();
      const int pos = min(sh.hit, m_n - 1);
      if (tid == pos) sh.scan[0] = in;
      __syncthreads();
      upto = sh.scan[0];
      cut_bin = min(cut_bin, bin);
      __syncthreads();
      return sh.sorted[pos];
    };
    Two sum;
    if (by_k) {
      cut = find(true, (uint32_t)top_k, {0.0f, 0.0f}, 0, sum);
    } else {
      uint64_t m = 0;
      if (lane < kBins)
        for (int r = 0; r < kC; ++r) m += sh.bins[r][lane].mass;
      sum = to_two(m, -kFrac - min(lane, kBins - 1));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum = add(sum, shfl_xor(sum, o));
    }
    if (by_p) cut = min(cut, find(false, 0, mul({fmaxf(top_p, 0.0f), 0.0f}, sum), 1, sum));
  }
  // ---- min-p: bins that it keeps whole, and those that it may cut
  int whole = cut_bin, last = cut_bin;  // bins whole .. last are looked at token by token
  if (by_m) {
    const float y = -lg2(min_p);
    whole = min(whole, max(0, (int)(y - 0.001f)));
    last = min(last, max(0, (int)(y + 0.001f)));
    if (whole >= kBins - 1) whole = min(cut_bin, kBins - 1);
  }
  const Two least = {min_p * kUp, 0.0f};
  // ---- kept mass and count of the runs
  auto stays = [&](float z, int i, Two w) {
    return rank_of(z, base + i) <= cut && (!by_m || base + i == best.at || !less(w, least));
  };
  Kept mine = {{0.0f, 0.0f}, 0};
  {
    uint64_t sum = 0;  // of 2^-54
    for (int b = 0; b < min(whole, kBins); ++b) {
      const uint64_t v = column[b * kT], m = v & ((1ull << kCount) - 1);
      mine.count += (int)(v >> kCount);
      const int s = 54 - kFrac - b;
      sum += s >= 0 ? m << s : (m + (1ull << (-s - 1))) >> -s;
    }
    mine.mass = to_two(sum, -54);
    if (whole < kBins) {
      for (int i = lo; i < hi; ++i) {
        const float z = at(i);
        if (!(z > -CUDART_INF_F)) continue;
        const int b = bin_of(y_of(z));
        if (b < whole || b > last) continue;
        Two w = weight2(z, M, c, sh.tab);
        if (!stays(z, i, w)) continue;
        ++mine.count;
        mine.mass = add(mine.mass, {w.h * (1.0f / kUp), w.l * (1.0f / kUp)});
      }
    }
  }
  const Two in = scan(mine.mass, lane);
  {
    const int n = __reduce_add_sync(kAll, mine.count);
    const Two m = shfl(in, 31);
    if (lane < kC) *remote(&sh.kept[rank * kW + warp], lane) = Kept{m, n};
  }
  sync();
  const Kept none = {{0.0f, 0.0f}, 0};
  const Kept k0 = e0 < kN ? sh.kept[e0] : none, k1 = e1 < kN ? sh.kept[e1] : none;
  if (rank == 0 && warp == 0 && a.kept) {
    const int n = __reduce_add_sync(kAll, k0.count + k1.count);
    if (lane == 0) a.kept[row] = n;
  }
  // ---- the draw: the warp, the lane, the token
  Two total = add(k0.mass, k1.mass);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total = add(total, shfl_xor(total, o));
  const Two goal = mul({us, 0.0f}, total);
  Two cum = {0.0f, 0.0f};
  const int chosen = pick(k0.mass, k1.mass, goal, cum, lane);
  if (chosen != rank * kW + warp) return;
  const unsigned reach = __ballot_sync(kAll, mine.mass.h > 0.0f && !less(add(cum, in), goal));
  const unsigned has = __ballot_sync(kAll, mine.mass.h > 0.0f);
  const int who = reach ? __ffs(reach) - 1 : 31 - __clz(has);
  if (who > 0) cum = add(cum, shfl(in, who - 1));
  const int start = __shfl_sync(kAll, lo, who), end = __shfl_sync(kAll, hi, who);
  int found = -1, last_in = -1;
  for (int i0 = start; i0 < end && found < 0; i0 += 32) {
    const int i = i0 + lane;
    Two w = {0.0f, 0.0f};
    if (i < end) {
      const float z = at(i);
      if (z > -CUDART_INF_F) {
        w = weight2(z, M, c, sh.tab);
        w = stays(z, i, w) ? Two{w.h * (1.0f / kUp), w.l * (1.0f / kUp)} : Two{0.0f, 0.0f};
      }
    }
    const Two s = add(cum, scan(w, lane));
    const unsigned h = __ballot_sync(kAll, w.h > 0.0f);
    const unsigned r = __ballot_sync(kAll, w.h > 0.0f && !less(s, goal));
    cum = shfl(s, 31);
    if (r) found = i0 + __ffs(r) - 1;
    if (h) last_in = i0 + 31 - __clz(h);
  }
  if (lane == 0) a.tokens[row] = found >= 0 ? base + found : last_in >= 0 ? base + last_in : best.at;
}

template <int kC>
Launched launch_c(const FilteredArgs& a, cudaStream_t s) {
  constexpr int kT = 256;
  constexpr int64_t kColumns = (int64_t)kBins * kT * 8, kMost = 200 * 1024;
  const int64_t each = ((a.V + kC * kT - 1) / (kC * kT)) | 1;
  int64_t smem = kColumns + std::min<int64_t>(a.V, kT * each) * 4;
  const int held = smem <= kMost;
  if (!held) smem = kColumns;
  static std::atomic<uint64_t> done{0};
  Launched l;
  l.error = allow_smem(k_sample_filtered<kC, kT>, (int)kMost, done);
  if (l.error != cudaSuccess) return l;
  if constexpr (kC == 1)
    l.add(launch_k(k_sample_filtered<1, kT>, dim3((unsigned)a.n), kT, smem, s, a, held));
  else
    l.add(launch_k_cluster(k_sample_filtered<kC, kT>, dim3((unsigned)a.n * kC), kT, smem, s, kC, a, held));
  return l;
}

}  // namespace

Launched launch_sample_filtered(const FilteredArgs& a, int sms, cudaStream_t s) {
  if (a.V > 4096) return launch_c<8>(a, s);
  return a.V > 2048 ? launch_c<4>(a, s) : launch_c<1>(a, s);
}

}  // namespace fsk
