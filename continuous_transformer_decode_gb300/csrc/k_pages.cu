// Page tables and slot maps (fs_pages_update): whole numbers only.
//
// Which pages a lane takes follows from two running sums: of the pages that the lanes
// want, in lane order, and of the free pages, in page order; the j-th wanted page is the
// j-th free one. Every block has the lanes' sums in shared memory (each forms them from
// the lanes' numbers, which are few) and a part of the pages; a thread finds the lane of a
// wanted page, of a page to let go or of a row by bisection there.
#include "fs_internal.h"

namespace fsk {
namespace {

constexpr int kT = 1024;
constexpr unsigned kAll = 0xffffffffu;

// Exclusive running sums over the block's threads of v; total becomes the sum.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* tmp, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(kAll, s, o);
    if (lane >= o) s += up;
  }
  if (lane == 31) tmp[warp] = s;
  __syncthreads();
  int64_t w = tmp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(kAll, w, o);
    if (lane >= o) w += up;
  }
  total = __shfl_sync(kAll, w, 31);
  const int64_t before = warp ? __shfl_sync(kAll, w, warp - 1) : 0;
  __syncthreads();
  return before + s - v;
}

// The last i < n with first[i] <= x (first[0] = 0 <= x; equal entries: the last).
__device__ __forceinline__ int owner(const int* first, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kT) k_pages(const PagesArgs a) {
  extern __shared__ int sh[];
  __shared__ int64_t tmp[32];
  const int n = a.n_lanes, tid = threadIdx.x;
  int* const held = sh;          // tokens kept
  int* const pages0 = sh + n;    // running sum of the pages wanted
  int* const rows0 = pages0 + n; // running sum of the rows (and first of the pages let go)
  pdl_wait();
  pdl_trigger();
  const int cap = a.max_pages * a.page_size, add = a.page_size - 1;
  auto pages_of = [&](int64_t tokens) { return (int)a.by_page.div((uint32_t)(tokens + add)); };
  const int each = (n + kT - 1) / kT, l0 = min(n, tid * each), l1 = min(n, l0 + each);
  int64_t gone_n;
  {
    int64_t mine = 0;
    for (int l = l0; l < l1; ++l) {
      const int had = max(0, min(a.lengths[l], cap));
      const int keep = a.keep ? max(0, a.keep[l]) : had;
      held[l] = min(had, keep);
      mine += pages_of(had) - pages_of(held[l]);
    }
    int64_t at = block_scan(mine, tmp, gone_n);
    for (int l = l0; l < l1; ++l) {
      rows0[l] = (int)at;
      at += pages_of(max(0, min(a.lengths[l], cap))) - pages_of(held[l]);
    }
  }
  __syncthreads();
  // ---- 1. pages let go
  for (int64_t t = tid; t < gone_n; t += kT) {
    const int l = owner(rows0, n, (int)t);
    int32_t* const e = a.table + (int64_t)l * a.max_pages + pages_of(held[l]) + ((int)t - rows0[l]);
    const int p = *e;
    *e = -1;
    if (p >= 0 && p < a.n_pages && atomicSub(a.holders + p, 1) <= 0) atomicAdd(a.holders + p, 1);
  }
  __syncthreads();
  // ---- what the lanes want
  int64_t want_n, rows_n;
  bool past = false;
  {
    int64_t want = 0, rows = 0;
    for (int l = l0; l < l1; ++l) {
      const int64_t g = max(0, a.grow[l]), end = held[l] + g;
      past |= end > cap;
      rows += g;
      if (end <= cap) want += pages_of(end) - pages_of(held[l]);
      else want += (end + add) / a.page_size - pages_of(held[l]);
    }
    int64_t at = block_scan(want, tmp, want_n), row = block_scan(rows, tmp, rows_n);
    for (int l = l0; l < l1; ++l) {
      const int64_t g = max(0, a.grow[l]), end = held[l] + g;
      pages0[l] = (int)at;
      rows0[l] = (int)row;
      at += end <= cap ? pages_of(end) - pages_of(held[l]) : 0;
      row += g;
    }
  }
  past = __syncthreads_or(past);
  // ---- free pages
  int64_t free_n = 0;
  {
    int64_t mine = 0;
    for (int p = tid; p < a.n_pages; p += kT) mine += __ldcg(a.holders + p) == 0;
    block_scan(mine, tmp, free_n);
  }
  const int code = past || want_n > free_n ? a.code_full : rows_n > a.max_rows ? a.code_rows : 0;
  const bool ok = code == 0;
  // ---- 2. the j-th free page is the j-th wanted
  if (ok) {
    int64_t rank0 = 0;
    for (int p0 = 0; p0 < a.n_pages && rank0 < want_n; p0 += kT) {
      const int p = p0 + tid;
      const bool is_free = p < a.n_pages && __ldcg(a.holders + p) == 0;
      int64_t found;
      const int64_t rank = rank0 + block_scan(is_free, tmp, found);
      if (is_free && rank < want_n) {
        const int l = owner(pages0, n, (int)rank);
        a.table[(int64_t)l * a.max_pages + pages_of(held[l]) + ((int)rank - pages0[l])] = p;
        a.holders[p] = 1;
      }
      rank0 += found;
    }
  }
  __syncthreads();
  // ---- 3. lanes and rows
  for (int l = tid; l < n; l += kT) {
    a.row_start[l] = ok ? rows0[l] : 0;
    if (l == 0) a.row_start[n] = ok ? (int)rows_n : 0;
    a.lengths[l] = held[l] + (ok ? max(0, a.grow[l]) : 0);
  }
  if (tid == 0) {
    const int64_t most = INT32_MAX;
    a.status[0] = code;
    a.status[1] = (int)min(rows_n, most);
    a.status[2] = (int)min(want_n, most);
    a.status[3] = (int)free_n;
  }
  const int rows = ok ? (int)rows_n : 0;
  for (int64_t r64 = tid; r64 < a.max_rows; r64 += kT) {
    const int r = (int)r64;
    int l = -1, pos = -1;
    int64_t slot = -1;
    if (r < rows) {
      l = owner(rows0, n, r);
      pos = held[l] + (r - rows0[l]);
      const int j = a.by_page.div((uint32_t)pos);
      if (a.row_slot)
        slot = (int64_t)a.table[(int64_t)l * a.max_pages + j] * a.page_size + (pos - j * a.page_size);
    }
    if (a.row_lane) a.row_lane[r] = l;
    if (a.row_position) a.row_position[r] = pos;
    if (a.row_length) a.row_length[r] = pos + 1;
    if (a.row_slot) a.row_slot[r] = slot;
  }
}

}  // namespace

Launched launch_pages(const PagesArgs& a, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  Launched l;
  l.error = allow_smem(k_pages, kMaxPageLanes * 12, done);
  if (l.error != cudaSuccess) return l;
  l.add(launch_k(k_pages, dim3(1), kT, (size_t)a.n_lanes * 12, s, a));
  return l;
}

}  // namespace fsk
