// Page tables and slot maps (fs_pages_update): whole numbers only.
//
// Which pages a lane takes follows from two running sums: of the pages that the lanes
// want, in lane order, and of the free pages, in page order; the j-th wanted page is the
// j-th free one. The lanes' sums are formed by every block for itself, in its shared
// memory, from the lanes' numbers, which are few; the pages are shared among the blocks of
// one cluster, which list their free ones and exchange the counts, and the wanted ones among
// all their threads. A page's or a row's lane is found by bisection in the running sums.
//
// The bytes are nothing (3 MB for 1021 lanes, 102282 pages and 131198 rows: 0.5 us); it is a
// chain of a few loads, sums and barriers: 5.2 us for one lane, 10 us for 256 lanes and 47955
// pages, 15 us for the 1021 lanes, 5 of them in the rows' kernel (by the cluster's eight SMs
// alone the rows took 11).
#include <cooperative_groups.h>

#include "fs_internal.h"

namespace fsk {
namespace {

namespace cg = cooperative_groups;

constexpr int kT = 1024, kW = kT / 32;
constexpr unsigned kAll = 0xffffffffu;
constexpr int kNew = -2;  // in place of a page: a lane that starts a new one, or takes nothing

// Words of 32 pages in a pool, which may have 2^31 - 1.
__host__ __device__ inline int page_words(int n_pages) { return (n_pages - 1) / 32 + 1; }

struct Three {
  int64_t a, b, c;
};
__device__ __forceinline__ Three operator+(Three x, Three y) { return {x.a + y.a, x.b + y.b, x.c + y.c}; }
__device__ __forceinline__ Three up(Three v, int o) {
  return {__shfl_up_sync(kAll, v.a, o), __shfl_up_sync(kAll, v.b, o), __shfl_up_sync(kAll, v.c, o)};
}
__device__ __forceinline__ Three at(Three v, int i) {
  return {__shfl_sync(kAll, v.a, i), __shfl_sync(kAll, v.b, i), __shfl_sync(kAll, v.c, i)};
}
__device__ __forceinline__ int up(int v, int o) { return __shfl_up_sync(kAll, v, o); }
__device__ __forceinline__ int at(int v, int i) { return __shfl_sync(kAll, v, i); }
// Inclusive running sums over the lanes of a warp.
template <typename T>
__device__ __forceinline__ T warp_scan(T v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = up(v, o);
    if (lane >= o) v = v + u;
  }
  return v;
}

// Exclusive running sums over the block's threads; total becomes the sum.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* tmp, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T s = warp_scan(v, lane);
  if (lane == 31) tmp[warp] = s;
  __syncthreads();
  const T w = warp_scan(tmp[lane], lane);
  total = at(w, 31);
  T before = at(w, max(warp - 1, 0));
  if (warp == 0) before = T{};
  T ahead = up(s, 1);
  if (lane == 0) ahead = T{};
  return before + ahead;
}

// The last i < n with first[i] <= x (first[0] = 0 <= x), in steps of `top` (the largest
// power of two below n) and halves of it: the same number of steps for every thread.
__device__ __forceinline__ int owner(const int* first, int n, int top, int x) {
  int lo = 0;
  for (int d = top; d > 0; d >>= 1)
    if (lo + d < n && first[lo + d] <= x) lo += d;
  return lo;
}

// What all lanes hold anyway, told to the compiler: a ballot or shuffle in a branch on it
// needs no reconvergence first.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(kAll, v, 0); }

// Rows from r0 on, four consecutive ones a thread: their lanes are looked for once, their
// numbers written in vectors. to_pos(l) takes a row of lane l to its token's place.
template <typename F>
__device__ __forceinline__ void write_rows(const PagesArgs& a, const int* rows0, int n, int top, int rows, int64_t r0,
                                           int64_t step, F to_pos) {
  const bool vec = ((reinterpret_cast<uintptr_t>(a.row_lane) | reinterpret_cast<uintptr_t>(a.row_position) |
                     reinterpret_cast<uintptr_t>(a.row_length) | reinterpret_cast<uintptr_t>(a.row_slot)) & 15) == 0;
  for (int64_t r64 = r0; r64 < a.rows_end; r64 += step) {
    const int r = (int)r64;
    int l[4], pos[4];
    int64_t slot[4];
    int own = r < rows ? owner(rows0, n, top, r) : 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const bool in = r64 + q < rows;
      if (q > 0 && in)
        while (own + 1 < n && rows0[own + 1] <= r + q) ++own;
      l[q] = in ? own : -1;
      pos[q] = in ? r + q + to_pos(own) : -1;
    }
    if (a.row_slot) {
      int page[4], j[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        j[q] = a.by_page.div((uint32_t)max(pos[q], 0));
        page[q] = l[q] >= 0 ? __ldcg(a.table + (int64_t)l[q] * a.max_pages + j[q]) : 0;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        slot[q] = l[q] >= 0 ? (int64_t)page[q] * a.page_size + (pos[q] - j[q] * a.page_size) : -1;
    }
    if (vec && r64 + 4 <= a.rows_end) {
      if (a.row_lane) *reinterpret_cast<int4*>(a.row_lane + r) = make_int4(l[0], l[1], l[2], l[3]);
      if (a.row_position) *reinterpret_cast<int4*>(a.row_position + r) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      if (a.row_length)
        *reinterpret_cast<int4*>(a.row_length + r) = make_int4(pos[0] + 1, pos[1] + 1, pos[2] + 1, pos[3] + 1);
      if (a.row_slot) {
        reinterpret_cast<longlong2*>(a.row_slot + r)[0] = make_longlong2(slot[0], slot[1]);
        reinterpret_cast<longlong2*>(a.row_slot + r)[1] = make_longlong2(slot[2], slot[3]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (r64 + q >= a.rows_end) break;
        if (a.row_lane) a.row_lane[r + q] = l[q];
        if (a.row_position) a.row_position[r + q] = pos[q];
        if (a.row_length) a.row_length[r + q] = pos[q] + 1;
        if (a.row_slot) a.row_slot[r + q] = slot[q];
      }
    }
  }
}

// kRows: with the rows; else another kernel writes them.
template <int kC, bool kRows>
__global__ void __launch_bounds__(kT) k_pages(const PagesArgs a) {
  extern __shared__ int sh[];
  __shared__ Three tmp3[kW];
  __shared__ int tmp[2][kW];
  __shared__ int2 free_of[8];  // the blocks' free pages, and how many of them are listed
  __shared__ int shared;       // a lane would grow into a page that others hold too
  static_assert(kC <= 8, "free_of");
  cg::cluster_group cluster = cg::this_cluster();
  auto sync = [&] {
    if constexpr (kC == 1) __syncthreads();
    else cluster.sync();
  };
  const int c = kC == 1 ? 0 : (int)cluster.block_rank();
  const int n = a.n_lanes, tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
  const int top = n > 1 ? 1 << (31 - __clz(n - 1)) : 0;
  int* const held = sh;           // tokens kept
  int* const pages0 = sh + n;     // running sum of the pages wanted
  int* const rows0 = pages0 + n;  // of the rows
  int* const gone0 = rows0 + n;   // of the pages let go
  uint16_t* const found = reinterpret_cast<uint16_t*>(gone0 + n);  // this block's free pages
  if (tid == 0) shared = 0;
  if constexpr (kC > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  pdl_wait();
  pdl_trigger();
  const int cap = a.max_pages * a.page_size, add = a.page_size - 1;
  auto pages_of = [&](int tokens) { return (int)a.by_page.div((uint32_t)(tokens + add)); };
  // ---- the lanes' running sums
  const int each = (n + kT - 1) / kT, l0 = min(n, tid * each), l1 = min(n, l0 + each);
  auto of_lane = [&](int l, int& keeps) {
    const int had = max(0, min(a.lengths[l], cap));
    keeps = a.keep ? min(had, max(0, a.keep[l])) : had;
    const int64_t grow = max(0, a.grow[l]), end = keeps + grow;
    const int first = pages_of(keeps);
    return Three{pages_of(had) - first, end <= cap ? pages_of((int)end) - first : (end + add) / a.page_size - first, grow};
  };
  // A lane grows into its last page, if that is not full, only where it alone holds it: a warp's
  // lanes are one block's to look at (by every block 1021 lanes took 1 us). The entry is asked
  // for here, its holders once pages have been let go, and both are looked at last.
  const bool looks = warp % kC == c;
  auto last_page = [&](int l, int keeps, int64_t grow) {  // -1: no page, or kNew
    const int j = a.by_page.div((uint32_t)keeps);
    return grow > 0 && keeps > j * a.page_size ? max(a.table[(int64_t)l * a.max_pages + j], -1) : kNew;
  };
  auto holders_or = [&](int p) {  // 1: the lane's own
    return p == kNew ? 1 : p >= 0 && p < a.n_pages ? __ldcg(a.holders + p) : 0;
  };
  bool past = false;
  int last = kNew;
  Three mine = {}, total;
  for (int l = l0; l < l1; ++l) {
    int keeps;
    const Three t = of_lane(l, keeps);
    past |= keeps + t.c > cap;
    held[l] = keeps;
    if (each == 1 && looks) last = last_page(l, keeps, t.c);
    mine = mine + t;
  }
  Three run = block_scan(mine, tmp3, total);
  if (each == 1) {
    if (l0 < l1) gone0[l0] = (int)run.a, pages0[l0] = (int)run.b, rows0[l0] = (int)run.c;
  } else {
    for (int l = l0; l < l1; ++l) {
      int keeps;
      const Three t = of_lane(l, keeps);
      gone0[l] = (int)run.a, pages0[l] = (int)run.b, rows0[l] = (int)run.c;
      run = run + t;
    }
  }
  past = __syncthreads_or(past);
  if constexpr (kC > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  // ---- 1. pages let go (past 2^31 of them the running sums do not count: lane by lane)
  if (total.a > 0) {
    auto let_go = [&](int l, int j) {
      int32_t* const e = a.table + (int64_t)l * a.max_pages + j;
      const int p = *e;
      *e = -1;
      if (p >= 0 && p < a.n_pages && atomicSub(a.holders + p, 1) <= 0) atomicAdd(a.holders + p, 1);
    };
    if (total.a <= INT32_MAX) {
      for (int64_t t = c * kT + tid; t < total.a; t += kC * kT) {
        const int l = owner(gone0, n, top, (int)t);
        let_go(l, pages_of(held[l]) + ((int)t - gone0[l]));
      }
    } else {
      for (int l = c; l < n; l += kC) {
        const int end = pages_of(max(0, min(a.lengths[l], cap)));
        for (int j = pages_of(held[l]) + tid; j < end; j += kT) let_go(l, j);
      }
    }
    sync();
  }
  // ---- free pages: this block's are page0 .. page1 - 1, 32 a warp's word
  const int words = page_words(a.n_pages);
  const int word0 = (int)((int64_t)words * c / kC), word1 = (int)((int64_t)words * (c + 1) / kC);
  auto holders_of = [&](int w, int end) {  // of the lane's page of a word
    const unsigned p = 32u * w + lane;
    return w < end && p < (unsigned)a.n_pages ? __ldcg(a.holders + p) : 1;
  };
  auto free_word = [&](int w, int end) { return __ballot_sync(kAll, holders_of(w, end) == 0); };
  // the first 1024 words, shared evenly by the warps, stay with the threads
  unsigned word = 0;
  const int share = min(32, (word1 - word0 + kW - 1) / kW), mine0 = word0 + warp * share;
  int alone = 1;
  for (int i0 = 0; i0 < max(share, 1); i0 += 8) {
    int h[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) h[i] = holders_of(mine0 + i0 + i, min(word1, mine0 + share));
    if (i0 == 0) alone = holders_or(last);  // the entry comes while these are on their way
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const unsigned m = __ballot_sync(kAll, h[i] == 0);
      if (i0 + i == lane) word = m;
    }
  }
  if (each > 1 && looks)
    for (int l = l0; l < l1; ++l)
      if (holders_or(last_page(l, held[l], a.grow[l])) != 1) alone = 0;
  int here;
  const int rank_in = block_scan(__popc(word), tmp[0], here);
  const int first_n = here;
  if (word1 - word0 > kT) {  // the same for the whole block
    int rest = 0, rest_n;
    for (int w = word0 + kT + warp; w < word1; w += kW) rest += __popc(free_word(w, word1));  // the same in all lanes
    block_scan(lane == 0 ? rest : 0, tmp[1], rest_n);
    here += rest_n;
  }
  for (int rank = rank_in; word; word &= word - 1)
    found[rank++] = (uint16_t)(32 * (mine0 - word0 + lane) + __ffs(word) - 1);
  if (tid < kC) *(kC == 1 ? &free_of[0] : cluster.map_shared_rank(&free_of[c], tid)) = make_int2(here, first_n);
  if (alone != 1)
    for (int b = 0; b < kC; ++b) *(kC == 1 ? &shared : cluster.map_shared_rank(&shared, b)) = 1;
  sync();
  int before = 0, free_n = 0;
  for (int b = 0; b < kC; ++b) {
    if (b == c) before = free_n;
    free_n += free_of[b].x;
  }
  const int code = past || total.b > free_n ? a.code_full : total.c > a.max_rows ? a.code_rows
                   : shared ? a.code_shared : 0;
  const bool ok = code == 0;
  // ---- 2. the j-th free page is the j-th wanted
  if (ok) {
    const int want = (int)total.b;
    auto take = [&](int p, int rank) {
      const int l = owner(pages0, n, top, rank);
      a.table[(int64_t)l * a.max_pages + pages_of(held[l]) + (rank - pages0[l])] = p;
      a.holders[p] = 1;
    };
    // the listed ones, shared by all threads of all blocks
#pragma unroll 2
    for (uint32_t at = c * kT + tid; at < (uint32_t)want; at += kC * kT) {  // want may be 2^31 - 1
      const int r = (int)at;
      int b = 0, i = r;
      while (b + 1 < kC && i >= free_of[b].x) i -= free_of[b++].x;
      if (i >= free_of[b].y) continue;
      const int at0 = (int)((int64_t)words * b / kC);
      take(32 * at0 + *(kC == 1 ? found + i : cluster.map_shared_rank(found + i, b)), r);
    }
    // and a block's own behind them
    int rank = before + first_n;
    for (int w0 = word0 + kT; w0 < word1 && rank < want; w0 += kW) {
      const int w = w0 + warp;
      const unsigned m = free_word(w, word1);
      int some;
      __syncthreads();
      const int ahead = block_scan(lane == 0 ? __popc(m) : 0, tmp[0], some);
      const int first = rank + at(ahead, 0);
      if ((m >> lane) & 1) {
        const int r = first + __popc(m & ((1u << lane) - 1));
        if (r < want) take(32 * w + lane, r);
      }
      rank += some;
    }
  }
  // ---- 3. lanes and rows
  sync();
  for (int l = c * kT + tid; l < n; l += kC * kT) {
    a.row_start[l] = ok ? rows0[l] : 0;
    a.lengths[l] = held[l] + (ok ? max(0, a.grow[l]) : 0);
  }
  if (c == 0 && tid == 0) {
    const int64_t most = INT32_MAX;
    a.row_start[n] = ok ? (int)total.c : 0;
    a.status[0] = code;
    a.status[1] = (int)min(total.c, most);
    a.status[2] = (int)min(total.b, most);
    a.status[3] = free_n;
  }
  if constexpr (kRows)
    write_rows(a, rows0, n, top, ok ? (int)total.c : 0, 4 * (int64_t)(c * kT + tid), 4 * kC * kT,
               [&](int l) { return held[l] - rows0[l]; });
}

// The rows alone, by many blocks, behind a call of the kernel above without them.
constexpr int kRowT = 256;
__global__ void __launch_bounds__(kRowT) k_page_rows(const PagesArgs a) {
  extern __shared__ int sh[];
  const int n = a.n_lanes, top = n > 1 ? 1 << (31 - __clz(n - 1)) : 0;
  pdl_wait();
  pdl_trigger();
  for (int l = threadIdx.x; l < n; l += kRowT) sh[l] = a.row_start[l];
  const int rows = a.row_start[n];
  __syncthreads();
  // lengths are the new ones: a lane's first token is its length less its rows
  write_rows(a, sh, n, top, rows, 4 * ((int64_t)blockIdx.x * kRowT + threadIdx.x), 4 * (int64_t)gridDim.x * kRowT,
             [&](int l) { return a.lengths[l] - (l + 1 < n ? sh[l + 1] : rows); });
}

template <int kC, bool kRows>
Launched launch_c(const PagesArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  Launched l;
  l.error = allow_smem(k_pages<kC, kRows>, kMaxPageLanes * 16 + 65536, done);
  if (l.error != cudaSuccess) return l;
  // four numbers a lane, and the places of a block's first 32768 pages
  const int64_t own = 32 * ((int64_t)page_words(a.n_pages) / kC + 1);
  const size_t smem = (size_t)a.n_lanes * 16 + (size_t)std::min<int64_t>(own, 32768) * 2;
  const bool fine = kC == 1 ? l.add(launch_k(k_pages<kC, kRows>, dim3(1), kT, smem, s, a))
                            : l.add(launch_k_cluster(k_pages<kC, kRows>, dim3(kC), kT, smem, s, kC, a));
  if (!kRows && fine) {
    const int64_t blocks = ((int64_t)a.rows_end + 4 * kRowT - 1) / (4 * kRowT);
    l.add(launch_k(k_page_rows, dim3((unsigned)std::min<int64_t>(blocks, 2048)), kRowT, (size_t)a.n_lanes * 4, s, a));
  }
  return l;
}

}  // namespace

// One block for small pools and batches, which saves the cluster's barriers; a kernel of its
// own for many rows. Without an array for them there are no rows to write, whatever their limit.
Launched launch_pages(PagesArgs a, cudaStream_t s) {
  a.rows_end = a.row_lane || a.row_position || a.row_length || a.row_slot ? a.max_rows : 0;
  if (a.n_pages <= 32768 && a.rows_end <= 4096 && a.n_lanes <= 1024) return launch_c<1, true>(a, s);
  return a.rows_end <= 16384 ? launch_c<8, true>(a, s) : launch_c<8, false>(a, s);
}

}  // namespace fsk
