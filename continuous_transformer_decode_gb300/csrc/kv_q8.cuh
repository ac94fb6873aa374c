// The 8-bit paged KV cache (include/fs.h, fs_kv_q8): device-side layout and
// the addressing shared by the kernels that write, read and attend to it.
#pragma once

#include "fs_internal.h"

namespace fsk {
namespace q8 {

// Slot (row index in [n_pages][Hkv][page_size]) of token t of `lane` for KV
// head g, or -1 when the lane, the token or the page-table entry is outside
// the cache: such a token holds nothing.
__device__ __forceinline__ int64_t slot_of(const KvQ8& c, int lane, int t, int g) {
  if ((unsigned)lane >= (unsigned)c.n_lanes || t < 0) return -1;
  const int pi = (int)c.by_page.div(t);
  if (pi >= c.max_pages) return -1;
  const int page = c.page_table[(int64_t)lane * c.max_pages + pi];
  if ((unsigned)page >= (unsigned)c.n_pages) return -1;
  return ((int64_t)page * c.Hkv + g) * c.page_size + (t - pi * c.page_size);
}

}  // namespace q8
}  // namespace fsk
