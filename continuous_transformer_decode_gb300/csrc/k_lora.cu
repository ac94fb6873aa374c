// Low-rank adapters of many requests (fs_lora_add): out = base + scale B (A x) with the
// row's own A [rank][K] and B [N][rank].
//
// The least it can do is to read base and x once, an adapter once for all its rows, and to
// write out. One launch does both products. Rows of any order are gathered out of windows of
// 256 by a hash of their adapters in shared memory; an item is up to kR rows of one adapter.
// Where items are few and large a cluster of eight or four blocks takes each: its blocks share K,
// exchange their parts of A x through distributed shared memory, and then share N. Else a block
// takes an item for itself, without barriers between blocks (the choice and its times are at
// launch_xy).
//
// Both products run on bf16 warp MMAs (m16n8k16, rows of x as M): a decode step has one to
// a few rows an adapter, so that most of a 128-row tcgen05 tile would be empty. Their rate here
// is 600 TFLOP/s (measured), so two parts of A x cost 8192 rows of 8 adapters, rank 64, 4096 to
// 14336, 57 us of MMAs, next to 79 us of bytes; they take 160 us. What bounds them is the
// warps' issue slots and their chains of shared loads, MMAs and stores (3.3 TB/s; MMAs active
// 0.4 of the time; one round of blocks, two an SM by their registers). Fragments of x and A
// come straight from global memory, 16 bytes a lane: the order of the summed index is free as
// long as both operands have the same, so a lane's 8 values of 32 feed two MMAs.
//
// Infinite weights. The parts of a value behind the first are 0 or of the other sign, which makes
// NaN of an infinite product. A sum that is NaN is therefore formed again: of A x (from f32 x)
// as the sum of its terms that are no finite numbers, of the columns with finite weights for
// the later parts. What finds them, a test of each chunk's results, takes 1 % of the 8192 rows'
// time and up to 3 % of others.
//
// A x is held in f32 and enters the second product as two bf16 parts (16 bits) for bf16
// results, which round by 2^-8 themselves, and three (24 bits) for f32 ones; an f32 x enters the
// first as three. Products of parts are exact, sums f32. Sums run over the same pieces in the
// same order however rows are tiled and shared: K in eight shares, each in eight pieces, so
// that a row's bits depend on the row alone.

#include <cooperative_groups.h>

#include <type_traits>

#include "attn_mma.cuh"
#include "fs_internal.h"

namespace fsk {
namespace {

namespace cg = cooperative_groups;

constexpr unsigned kAll = 0xffffffffu;
constexpr int kShares = 8, kT = 256, kW = kT / 32;  // shares of K, threads, warps
constexpr int kWindow = kT;                         // rows that are gathered, one a thread
constexpr int kSlots = 2 * kWindow;

// Three bf16 parts of f32 values that hold their 24 bits (two: 16). A value past bf16's
// range is its largest, and the rest; infinities and NaN are in the first part alone.
template <int kParts>
__device__ __forceinline__ void split(float x, __nv_bfloat16 (&p)[kParts]) {
  __nv_bfloat16 h = __float2bfloat16_rn(x);
  float f = __bfloat162float(h);
  if (fabsf(f) > 3.3895314e38f) {  // inf or NaN
    if (fabsf(x) <= 3.4028235e38f) {
      h = __ushort_as_bfloat16(x < 0 ? 0xff7f : 0x7f7f);
      f = __bfloat162float(h);
    } else {
      f = x = 0.0f;
    }
  }
  p[0] = h;
  float rest = x - f;
#pragma unroll
  for (int i = 1; i < kParts; ++i) {
    p[i] = __float2bfloat16_rn(rest);
    rest -= __bfloat162float(p[i]);
  }
}

// 8 consecutive values as bf16 parts.
template <typename T>
struct Eight {
  static constexpr int kParts = sizeof(T) == 4 ? 3 : 1;
  uint4 p[kParts];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kParts; ++i) p[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void load(const T* x, bool vec) {
    if constexpr (sizeof(T) == 2) {
      if (vec) {
        p[0] = *reinterpret_cast<const uint4*>(x);
      } else {
        const uint16_t* u = reinterpret_cast<const uint16_t*>(x);
        uint32_t* w = reinterpret_cast<uint32_t*>(&p[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = (uint32_t)u[2 * i] | ((uint32_t)u[2 * i + 1] << 16);
      }
    } else {
      float v[8];
      if (vec) {
        const float4 a = reinterpret_cast<const float4*>(x)[0], b = reinterpret_cast<const float4*>(x)[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
        v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = x[i];
      }
      parts(v);
    }
  }
  __device__ __forceinline__ void parts(const float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
      __nv_bfloat16* out[3] = {reinterpret_cast<__nv_bfloat16*>(&p[0]), reinterpret_cast<__nv_bfloat16*>(&p[1]),
                               reinterpret_cast<__nv_bfloat16*>(&p[2])};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        __nv_bfloat16 s[3];
        split(v[i], s);
        out[0][i] = s[0], out[1][i] = s[1], out[2][i] = s[2];
      }
    }
  }
};

// d += a b over 16 of 32 values of the summed index (half 0, then 1): rows g (lo) and g + 8
// (hi) of a, column g of b, a lane's 8 values each. Products that do not add to the same sums
// go between the halves: an MMA waits for the last one's sums.
__device__ __forceinline__ void mma_half(float (&d)[4], const uint4& lo, const uint4& hi, const uint4& b, int half) {
  const uint32_t a[4] = {half ? lo.z : lo.x, half ? hi.z : hi.x, half ? lo.w : lo.y, half ? hi.w : hi.y};
  attn::mma16816(d, a, half ? b.z : b.x, half ? b.w : b.y);
}

// 8 consecutive values as they lie in memory.
template <typename T>
struct Raw8 {
  static constexpr int kV = sizeof(T) / 2;
  uint4 v[kV];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kV; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  // the first n of p (whole: all 8, 16-byte aligned)
  __device__ __forceinline__ void load(const T* p, bool whole, int n) {
    if (whole) {
#pragma unroll
      for (int i = 0; i < kV; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
      clear();
      T* t = reinterpret_cast<T*>(v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) t[i] = p[i];
    }
  }
  __device__ __forceinline__ void store(T* p, bool whole, int n) const {
    if (whole) {
#pragma unroll
      for (int i = 0; i < kV; ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
    } else {
      const T* t = reinterpret_cast<const T*>(v);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = t[i];
    }
  }
  // What the sums of values 2 i and 2 i + 1 start with, and their end. f32 values are added
  // last, so that the sums of products do not round at the size of base; bf16 ones, which round
  // to 8 bits themselves, first.
  __device__ __forceinline__ void start(int i, float& a, float& b) const {
    if constexpr (sizeof(T) == 4) {
      a = b = 0.0f;
    } else {
      const uint32_t u = reinterpret_cast<const uint32_t*>(v)[i];
      a = __uint_as_float(u << 16), b = __uint_as_float(u & 0xffff0000u);
    }
  }
  // NaN where m or one of the values is (and for some that are past half their type's range).
  __device__ __forceinline__ uint32_t any_nan(uint32_t m) const {
    if constexpr (sizeof(T) == 4) {
      const float* f = reinterpret_cast<const float*>(v);
      return __float_as_uint(fmaf(fmaf(f[0], f[1], f[2]), fmaf(f[3], f[4], f[5]), fmaf(f[6], f[7], __uint_as_float(m))));
    } else {
      const __nv_bfloat162* f = reinterpret_cast<const __nv_bfloat162*>(v);
      __nv_bfloat162 r = __hfma2(__hfma2(f[0], f[1], f[2]), f[3], *reinterpret_cast<const __nv_bfloat162*>(&m));
      return *reinterpret_cast<uint32_t*>(&r);
    }
  }
  static __device__ __forceinline__ bool is_nan(uint32_t m) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(m) != __uint_as_float(m);
    else return !__hbeq2(*reinterpret_cast<const __nv_bfloat162*>(&m), *reinterpret_cast<const __nv_bfloat162*>(&m));
  }
  __device__ __forceinline__ void end(int i, float a, float b) {
    if constexpr (sizeof(T) == 4) {
      float* f = reinterpret_cast<float*>(v);
      f[2 * i] += a, f[2 * i + 1] += b;
    } else {
      reinterpret_cast<uint32_t*>(v)[i] = attn::pack_bf16(a, b);
    }
  }
};

struct Gather {
  int key[kSlots];
  uint16_t count[kW][kSlots];  // rows of a warp
  int id[kWindow];
  int16_t nth[kWindow];   // of its adapter's rows in the window
  int16_t lead[kWindow];  // first rows of the items
  int row[32];            // of an item
  int firsts[kW], bare[kW];
};

// Shared memory behind Gather: the parts of A x, and f32 tiles of sums, a warp's for each of
// the block's shares and, in a cluster, a share's each; the warps' buffers of B lie where the sums were. A part of
// a row tile is a run of MMA fragments, [block of 32 ranks][half][lane] of 16 bytes, so that one
// load gives a lane the four registers of an operand, side by side.
struct Sizes {
  int tile;  // bytes of a part of a row tile
  int64_t low, bytes;
  __host__ __device__ Sizes(int mt, int item_blocks, int parts, int rank) {
    tile = (rank + 31) / 32 * 1024;
    low = (int64_t)parts * mt * tile;
    const int tiles = item_blocks == 1 ? kW : kShares / item_blocks * kW + kShares;
    const int64_t sums = (int64_t)tiles * mt * 16 * rank * 4, buffers = (int64_t)kW * 128 * rank;
    bytes = (int64_t)((sizeof(Gather) + 15) / 16 * 16) + low + (sums > buffers ? sums : buffers);
  }
};

__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
// 16 bytes to shared memory, zeros without `in`.
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
}

// The sum of n terms of which some are infinite or NaN (NaN where none is).
template <typename F>
__device__ __forceinline__ float sum_of(int n, F term) {
  float s = 0.0f;
#pragma unroll 1
  for (int i = 0; i < n && s == s; ++i) {
    const float t = term(i);
    if (!(fabsf(t) <= 3.4028235e38f)) s += t;
  }
  return s != 0.0f ? s : __int_as_float(0x7fffffff);
}

// Two weights without infinities and NaN (0 in their place), for the parts of a value behind the
// first.
__device__ __forceinline__ uint32_t finite2(uint32_t w) { return w & __vcmpltu2(w & 0x7fff7fffu, 0x7f807f80u); }
__device__ __forceinline__ uint4 finite8(const uint4& w) {
  return make_uint4(finite2(w.x), finite2(w.y), finite2(w.z), finite2(w.w));
}

// What all lanes hold anyway, told to the compiler: inside a branch or loop on it MMAs and
// shuffles then need no reconvergence before each of them.
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(kAll, v, 0); }

// kMT: row tiles of an item; kBlocks: blocks that take one together, 8 or 4 (a cluster) or 1,
// whose warps have a share of K each.
template <typename TX, typename TY, int kMT, int kBlocks>
__global__ void __launch_bounds__(kT, 2) k_lora(const LoraArgs a, int per_window) {
  constexpr int kR = 16 * kMT;                  // rows of an item
  constexpr int kMP = kMT == 1 || sizeof(TY) == 4 ? 1 : 2;  // row tiles at a time
  constexpr int kParts = sizeof(TY) == 4 ? 3 : 2;
  extern __shared__ __align__(16) unsigned char dyn[];
  Gather& sh = *reinterpret_cast<Gather*>(dyn);
  constexpr bool kSolo = kBlocks == 1;
  const Sizes sz(kMT, kBlocks, kParts, a.rank);
  unsigned char* const low = dyn + (sizeof(Gather) + 15) / 16 * 16;
  float* const sums = reinterpret_cast<float*>(low + sz.low);
  cg::cluster_group cluster = cg::this_cluster();
  static_assert(kW == kShares, "a warp a share of K");
  const int c = kSolo ? 0 : (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31, g = lane >> 2, tig = lane & 3;
  // the other blocks' shared memory can be written once they have started
  if constexpr (!kSolo) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  for (int i = tid; i < kSlots; i += kT) sh.key[i] = -1;
  for (int i = tid; i < kW * kSlots / 8; i += kT) reinterpret_cast<uint4*>(sh.count)[i] = make_uint4(0, 0, 0, 0);
  pdl_wait();
  pdl_trigger();
  const int item0 = blockIdx.x / kBlocks % per_window;
  const int first = (int)(blockIdx.x / kBlocks / per_window) * kWindow;
  // ---- the window's rows by adapter
  const int my_row = first + tid;
  const int my_id = my_row < a.n ? a.adapter[my_row] : -1;
  const bool has = my_id >= 0 && my_id < a.n_adapters;
  __syncthreads();
  int slot = 0;
  if (has) {
    slot = (int)((uint32_t)my_id * 2654435761u >> 23);
    static_assert(kSlots == 512, "nine bits");
    while (true) {
      const int old = atomicCAS(&sh.key[slot], -1, my_id);
      if (old == -1 || old == my_id) break;
      slot = (slot + 1) % kSlots;
    }
  }
  const unsigned same = __match_any_sync(kAll, has ? my_id : -1);
  const unsigned below = (1u << lane) - 1;
  if (has && (same & below) == 0) sh.count[warp][slot] = (uint16_t)__popc(same);
  sh.id[tid] = has ? my_id : -1;
  __syncthreads();
  int nth = __popc(same & below);
  if (has)
    for (int w = 0; w < warp; ++w) nth += sh.count[w][slot];
  sh.nth[tid] = (int16_t)nth;
  const unsigned leads = __ballot_sync(kAll, has && nth % kR == 0);
  const unsigned bare = __ballot_sync(kAll, !has && my_row < a.n);
  if (lane == 0) sh.firsts[warp] = __popc(leads), sh.bare[warp] = __popc(bare);
  __syncthreads();
  int items = 0, bares = 0, at = 0, bare_at = 0;
#pragma unroll
  for (int w = 0; w < kW; ++w) {
    if (w == warp) at = items, bare_at = bares;
    items += sh.firsts[w];
    bares += sh.bare[w];
  }
  items = uniform(items);
  if (has && nth % kR == 0) sh.lead[at + __popc(leads & below)] = (int16_t)tid;

  // this block's columns, in chunks of 32
  const int chunks = (a.N + 31) / 32, per = (chunks + kBlocks - 1) / kBlocks;
  const int chunk0 = min(chunks, c * per), chunk1 = min(chunks, chunk0 + per);
  const TX* const x = static_cast<const TX*>(a.x);
  const TY* const base = static_cast<const TY*>(a.base);
  TY* const out = static_cast<TY*>(a.out);
  const bool x_vec = (reinterpret_cast<uintptr_t>(x) & 15) == 0 && a.x_stride * sizeof(TX) % 16 == 0;
  const bool y_vec = ((reinterpret_cast<uintptr_t>(base) | reinterpret_cast<uintptr_t>(out)) & 15) == 0 &&
                     (a.base_stride | a.out_stride) * sizeof(TY) % 16 == 0;
  if constexpr (!kSolo) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  // ---- K, in blocks of 32: eight shares of eight pieces each
  constexpr int kOwn = kSolo ? 1 : kShares / kBlocks;  // shares of a block (kSolo: of a warp)
  const int kbs = (a.K + 31) / 32, share0 = kSolo ? warp : c * kOwn;
  const int tiles = a.rank / 8, rblocks = (a.rank + 31) / 32;
  auto piece = [&](int q, int s) {  // the s-th of own share q starts here
    const int kb0 = (int)((int64_t)kbs * (share0 + q) / kShares), kb1 = (int)((int64_t)kbs * (share0 + q + 1) / kShares);
    return kb0 + (kb1 - kb0) * s / kW;
  };

  for (int item = item0; item < items; item += per_window) {
    __syncthreads();  // also: sh.lead
    const int lead = uniform(sh.lead[item]), id = uniform(sh.id[lead]), part = sh.nth[lead] / kR;
    const bool mine = has && my_id == id && nth / kR == part;
    if (mine) sh.row[nth % kR] = my_row;
    const int rows = uniform(__syncthreads_count(mine));
    const float scale = a.scale[id];
    const __nv_bfloat16* const A = a.A + (int64_t)id * a.rank * a.K;
    const __nv_bfloat16* const B = a.B + (int64_t)id * a.N * a.rank;
    auto row_of = [&](int i) { return i < rows ? sh.row[i] : -1; };
    if constexpr (!kSolo)
      if (item != item0) cluster.sync();  // the last item's sums and columns are done with

    auto put = [&](float* to, int mt, int nt, const float (&d)[4]) {
      float* p = to + (16 * mt + g) * a.rank + 8 * nt + 2 * tig;
      *reinterpret_cast<float2*>(p) = make_float2(d[0], d[1]);
      *reinterpret_cast<float2*>(p + 8 * a.rank) = make_float2(d[2], d[3]);
    };
    const int tile = kMT * 16 * a.rank;
    {
      int64_t r0[kMT], r1[kMT];
#pragma unroll
      for (int m = 0; m < kMT; ++m) r0[m] = row_of(16 * m + g), r1[m] = row_of(16 * m + g + 8);
      for (int nt0 = 0; nt0 < tiles; nt0 += 4) {  // four tiles of ranks
        // d += x A^T over blocks b0 .. b1 - 1 of K
        auto product = [&](int b0, int b1, float (&d)[kMT][4][4]) {
#pragma unroll 2
          for (int b = b0; b < b1; ++b) {
            const int k = 32 * b + 8 * tig;
            const bool in = k < a.K;
            Eight<TX> lo[kMT], hi[kMT];
#pragma unroll
            for (int m = 0; m < kMT; ++m) {
              lo[m].clear(), hi[m].clear();
              if (in && r0[m] >= 0) lo[m].load(x + r0[m] * a.x_stride + k, x_vec);
              if (in && r1[m] >= 0) hi[m].load(x + r1[m] * a.x_stride + k, x_vec);
            }
            uint4 w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              w[j] = in && nt0 + j < tiles ? *reinterpret_cast<const uint4*>(A + (int64_t)(8 * (nt0 + j) + g) * a.K + k)
                                           : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 2 * Eight<TX>::kParts; ++i)
#pragma unroll
              for (int m = 0; m < kMT; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) mma_half(d[m][j], lo[m].p[i / 2], hi[m].p[i / 2], w[j], i % 2);
          }
        };
        float d[kOwn][kMT][4][4] = {};
        if constexpr (kSolo) {  // the warp's share, piece by piece
          product(piece(0, 0), piece(0, 1), d[0]);
          for (int p = 1; p < kW; ++p) {
            float e[kMT][4][4] = {};
            product(piece(0, p), piece(0, p + 1), e);
#pragma unroll
            for (int m = 0; m < kMT; ++m)
#pragma unroll
              for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) d[0][m][j][q] += e[m][j][q];
          }
        } else {  // the warp's piece of the block's shares
#pragma unroll
          for (int q = 0; q < kOwn; ++q) product(piece(q, warp), piece(q, warp + 1), d[q]);
        }
#pragma unroll
        for (int q = 0; q < kOwn; ++q)
#pragma unroll
          for (int m = 0; m < kMT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (nt0 + j < tiles) put(sums + (q * kW + warp) * tile, m, nt0 + j, d[q][m][j]);
      }
      __syncthreads();
      if constexpr (!kSolo) {
        for (int i = tid; i < kOwn * tile; i += kT) {
          const int q = kOwn == 1 ? 0 : i / tile, at = i - q * tile;
          const float* const p = sums + q * kW * tile + at;
          float s = p[0];
#pragma unroll
          for (int w = 1; w < kW; ++w) s += p[w * tile];
          for (int r = 0; r < kBlocks; ++r)
            *cluster.map_shared_rank(sums + (kOwn * kW + share0 + q) * tile + at, r) = s;
        }
        cluster.sync();
      }
      // a value of A x a thread and step: its fragment's lane and half, two ranks a register
      for (int i = tid; i < kMT * 16 * 32 * rblocks; i += kT) {
        const int m = i / (32 * rblocks), r = i - m * 32 * rblocks;
        float v = 0.0f;
        if (r < a.rank) {
          const float* p = sums + (kSolo ? 0 : kOwn * kW) * tile + m * a.rank + r;
          v = p[0];
#pragma unroll
          for (int b = 1; b < kShares; ++b) v += p[b * tile];
          if (sizeof(TX) == 4 && v != v && m < rows) {  // of parts of x: an infinity of A?
            const TX* const xr = x + sh.row[m] * a.x_stride;
            const __nv_bfloat16* const Ar = A + (int64_t)r * a.K;
            v = sum_of(a.K, [&](int k) { return (float)xr[k] * __bfloat162float(Ar[k]); });
          }
          v *= scale;
        }
        __nv_bfloat16 u[kParts];
        split(v, u);
        const int unit = ((r >> 5) * 2 + ((r >> 2) & 1)) * 32 + (m & 7) * 4 + ((r >> 3) & 3);
        const int reg = ((r >> 1) & 1) * 2 + ((m >> 3) & 1);
        unsigned char* const to = low + (m >> 4) * sz.tile + unit * 16 + reg * 4 + (r & 1) * 2;
#pragma unroll
        for (int p = 0; p < kParts; ++p) *reinterpret_cast<__nv_bfloat16*>(to + p * kMT * sz.tile) = u[p];
      }
      __syncthreads();
    }
    // ---- the columns: chunks of 32, a lane's 8 consecutive ones from four MMA tiles. B comes
    // by two buffers of the warp's own, base of the next tiles is asked for before the
    // products of these. 16-byte parts of odd columns are swapped where a column is 128 bytes
    // long or twice that, so that a quarter of a warp reads all banks.
    // What does not change from chunk to chunk is formed once (in all, a chunk of two row tiles at
    // rank 64 took 1150 instructions without that; its MMAs are 64).
    const int swap = a.rank % 64 ? 0 : 4;
    const uint32_t buffers = attn::smem_u32(sums) + warp * 128 * a.rank;
    const uint32_t b_to = buffers + 16 * (lane ^ ((lane / tiles) & 1) * swap);  // 32 / tiles is even or swap 0
    const int b_end = a.N * tiles;                                              // 16-byte parts of B
    const uint32_t b_at = buffers + (8 * (g >> 1) + (g & 1)) * 16 * tiles;      // column g of MMA tile 0
    const uint32_t t_at = attn::smem_u32(low) + 16 * lane;
    int row[kMT][2];
#pragma unroll
    for (int m = 0; m < kMT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) row[m][h] = row_of(16 * m + g + 8 * h);
    const int some_row = sh.row[0];  // read in place of none
    auto fetch = [&](int chunk, int slot) {
      if (chunk < chunk1) {
        const int i0 = 32 * chunk * tiles + lane;
        const uint32_t to = b_to + slot * 64 * a.rank;
        const __nv_bfloat16* const from = B + (int64_t)8 * i0;
#pragma unroll 4
        for (int k = 0; k < tiles; ++k) {
          const bool in = i0 + 32 * k < b_end;
          copy16(to + 512 * k, in ? from + 256 * k : B, in);
        }
      }
      attn::cp_commit();
    };
    Raw8<TY> next[kMP][2];
    auto ask = [&](int chunk, auto m0) {
      if (!base || chunk >= chunk1) return;
      const int col = 32 * chunk + 8 * tig;
      const bool whole = y_vec && 32 * chunk + 32 <= a.N;
#pragma unroll
      for (int m = 0; m < kMP; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = row[decltype(m0)::value + m][h];
          next[m][h].load(base + (r >= 0 ? r : some_row) * a.base_stride + col, whole, a.N - col);
        }
    };
#pragma unroll
    for (int m = 0; m < kMP; ++m) next[m][0].clear(), next[m][1].clear();  // without base
    using First = std::integral_constant<int, 0>;
    using Second = std::integral_constant<int, kMT - kMP>;
    fetch(chunk0 + warp, 0);
    ask(chunk0 + warp, First{});
    int slot = 0;
    // The same sums in the same order, with finite weights for the later parts of A x.
    auto redo = [&](auto m0, int col, int slot, auto& y) {
      constexpr int kM = decltype(m0)::value;
      const bool whole = y_vec && (col & ~31) + 32 <= a.N;
#pragma unroll
      for (int m = 0; m < kMP; ++m) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = row[kM + m][h];
          if (base) y[m][h].load(base + (r >= 0 ? r : some_row) * a.base_stride + col, whole, a.N - col);
          else y[m][h].clear();
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float d[4];
#pragma unroll
          for (int h = 0; h < 2; ++h) y[m][h].start(j, d[2 * h], d[2 * h + 1]);
#pragma unroll 1
          for (int b = 0; b < rblocks; ++b) {
            const int q = 4 * b + tig;
            uint4 w = q < tiles ? lds128(b_at + slot * 64 * a.rank + 16 * (q ^ (g & 1) * swap) + 32 * j * tiles)
                                : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
              if (p == 1) w = finite8(w);
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint4 f = lds128(t_at + (p * kMT + kM + m) * sz.tile + 1024 * b + 512 * i);
                const uint32_t x[4] = {f.x, f.y, f.z, f.w};
                attn::mma16816(d, x, i ? w.z : w.x, i ? w.w : w.y);
              }
            }
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) y[m][h].end(j, d[2 * h], d[2 * h + 1]);
        }
      }
    };
    for (int chunk = chunk0 + warp; chunk < chunk1; chunk += kW, slot ^= 1) {
      fetch(chunk + kW, slot ^ 1);
      attn::cp_wait<1>();
      __syncwarp();
      const int col = 32 * chunk + 8 * tig;
      const bool whole = y_vec && 32 * chunk + 32 <= a.N;
      auto columns = [&](auto m0, auto then) {
        constexpr int kM = decltype(m0)::value;
        Raw8<TY> y[kMP][2];
        float d[kMP][4][4];
        uint32_t nan = 0;
#pragma unroll
        for (int m = 0; m < kMP; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (sizeof(TY) == 4) y[m][h] = next[m][h];
#pragma unroll
            for (int j = 0; j < 4; ++j) next[m][h].start(j, d[m][j][2 * h], d[m][j][2 * h + 1]);
          }
        then();
        uint32_t t = t_at + kM * sz.tile;
        const uint32_t w_at = b_at + slot * 64 * a.rank;
#pragma unroll 1
        for (int b = 0; b < rblocks; ++b, t += 1024) {
          uint4 w[4];  // tile j's column g
          const int q = 4 * b + tig;
          const uint32_t at = w_at + 16 * (q ^ (g & 1) * swap);
#pragma unroll
          for (int j = 0; j < 4; ++j) w[j] = q < tiles ? lds128(at + 32 * j * tiles) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int p = 0; p < kParts; ++p) {
            uint4 f[kMP][2];
#pragma unroll
            for (int m = 0; m < kMP; ++m)
#pragma unroll
              for (int i = 0; i < 2; ++i) f[m][i] = lds128(t + (p * kMT + m) * sz.tile + 512 * i);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int m = 0; m < kMP; ++m)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const uint32_t x[4] = {f[m][i].x, f[m][i].y, f[m][i].z, f[m][i].w};
                  attn::mma16816(d[m][j], x, i ? w[j].z : w[j].x, i ? w[j].w : w[j].y);
                }
          }
        }
#pragma unroll
        for (int m = 0; m < kMP; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int j = 0; j < 4; ++j) y[m][h].end(j, d[m][j][2 * h], d[m][j][2 * h + 1]);
            nan = y[m][h].any_nan(nan);
          }
        if (__any_sync(kAll, Raw8<TY>::is_nan(nan))) redo(m0, col, slot, y);
#pragma unroll
        for (int m = 0; m < kMP; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (row[kM + m][h] >= 0) y[m][h].store(out + row[kM + m][h] * a.out_stride + col, whole, a.N - col);
      };
      if (kMT == kMP || rows <= 16 * kMP) {
        columns(First{}, [&] { ask(chunk + kW, First{}); });
      } else {
        columns(First{}, [&] { ask(chunk, Second{}); });
        columns(Second{}, [&] { ask(chunk + kW, First{}); });
      }
      __syncwarp();  // before the buffer is filled again
    }
    attn::cp_wait<0>();
  }
  // ---- rows without an adapter, shared by the window's clusters
  if (a.base != a.out && bares) {
    unsigned m = bare;
    for (int i = bare_at; m; ++i, m &= m - 1) {  // a warp its own rows
      if (i % per_window != item0) continue;
      const int64_t row = first + warp * 32 + __ffs(m) - 1;
      for (int j = 32 * chunk0 + 8 * lane; j < min(a.N, 32 * chunk1); j += 256) {
        const bool whole = y_vec && j + 8 <= a.N;
        Raw8<TY> v;
        v.clear();
        if (base) v.load(base + row * a.base_stride + j, whole, a.N - j);
        v.store(out + row * a.out_stride + j, whole, a.N - j);
      }
    }
  }
}

template <typename TX, typename TY, int kMT, int kBlocks>
Launched launch_t(const LoraArgs& a, int64_t per_window, cudaStream_t s) {
  constexpr int kParts = sizeof(TY) == 4 ? 3 : 2;
  auto kernel = k_lora<TX, TY, kMT, kBlocks>;
  static std::atomic<uint64_t> done{0};
  Launched l;
  l.error = allow_smem(kernel, (int)Sizes(kMT, kBlocks, kParts, 128).bytes, done);
  if (l.error != cudaSuccess) return l;
  const int per = (int)std::min<int64_t>(std::min(a.n, kWindow), std::max<int64_t>(1, per_window));
  const dim3 grid((unsigned)((a.n + (int64_t)kWindow - 1) / kWindow * per * kBlocks));
  const size_t smem = (size_t)Sizes(kMT, kBlocks, kParts, a.rank).bytes;
  if constexpr (kBlocks == 1) l.add(launch_k(kernel, grid, kT, smem, s, a, per));
  else l.add(launch_k_cluster(kernel, grid, kT, smem, s, kBlocks, a, per));
  return l;
}

// How many blocks take an item, from how long it would take at most, as the adapters' mix is
// not known here: a window of 256 rows has up to n_adapters items and one more for every 16
// rows. A block by itself takes 6 us and `alone`, four together 4.7 us and a quarter of it, eight
// 4 us and an eighth; 2 blocks an SM run at a time. Measured, us, by 1 | 4 | 8 blocks (rows
// in any order, adapters, rank, K, N; bf16):
//   30, 8, 64, 4096, 14336: 60 | 21 | 16      100, 64, 16, 4096, 4096: 18 | 9.8 | 13
//   100, 200, 16, 576, 960: 7.0 | 11 | 17     256, 8, 16, 4096, 4096: 21 | 9.0 | 7.2
//   256, 64, 16, 4096, 4096: 24 | 11 | 14     256, 200, 16, 576, 960: 8.8 | 12 | 26
//   1000, 8, 64, 4096, 14336: 93 | 55 | 53    1000, 64, 16, 4096, 4096: 26 | 49 | 52
//   2500, 8, 64, 4096, 14336: 98 | 99 | 121   8192, 64, 16, 4096, 4096: 191 | 303 | 389
// An item takes two row tiles where adapters have 256 rows and more (8192 rows of 64 in any order,
// rank 16, 4096 to 4096: 279 | 191 by two | one) and items of one tile are more than run at a
// time, which 8 adapters have from 4737 rows on. Rows in runs, blocks alone, 8, 16, 4096, 4096 and
// 8, 64, 4096, 14336:
//   4097 rows: 45 | 34, 157 | 101    4700: 46 | 39, 157 | 105    4864: 47 | 57, 158 | 163
//   5300 rows: 47 | 60, 158 | 176    6000: 47 | 61, 158 | 187    8192: 50 | 64, 161 | 195
template <typename TX, typename TY>
Launched launch_xy(const LoraArgs& a, int sms, cudaStream_t s) {
  const int64_t windows = (a.n + (int64_t)kWindow - 1) / kWindow;
  const int64_t items = std::min<int64_t>(a.n, windows * std::min<int64_t>(kWindow, (int64_t)a.n_adapters + kWindow / 16));
  const double alone = a.N / 256.0 * (0.5 + 0.007 * a.rank) + a.K / 1024.0;
  auto estimate = [&](int blocks, double start) {
    const int64_t at_once = std::max(1, 2 * sms / blocks);
    return (double)((items + at_once - 1) / at_once) * (start + alone / blocks);
  };
  const double by_8 = estimate(8, 4), by_4 = estimate(4, 4.7), by_1 = estimate(1, 6);
  if (by_8 <= by_4 && by_8 <= by_1) return launch_t<TX, TY, 1, 8>(a, 2 * sms / 8 / windows, s);
  if (by_4 <= by_1) return launch_t<TX, TY, 1, 4>(a, 2 * sms / 4 / windows, s);
  // four blocks an SM in all, at least eight a window
  const int64_t each = std::max<int64_t>(8, 4 * sms / windows);
  if (((int64_t)a.n + 15) / 16 + a.n_adapters > 2 * sms && a.n / 256 >= a.n_adapters) return launch_t<TX, TY, 2, 1>(a, each, s);
  return launch_t<TX, TY, 1, 1>(a, each, s);
}

}  // namespace

Launched launch_lora(const LoraArgs& a, int x_type, int y_type, int sms, cudaStream_t s) {
  if (x_type == X_F32)
    return y_type == X_F32 ? launch_xy<float, float>(a, sms, s) : launch_xy<float, __nv_bfloat16>(a, sms, s);
  return y_type == X_F32 ? launch_xy<__nv_bfloat16, float>(a, sms, s)
                         : launch_xy<__nv_bfloat16, __nv_bfloat16>(a, sms, s);
}

}  // namespace fsk
