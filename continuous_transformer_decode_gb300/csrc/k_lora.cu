// Low-rank adapters of many requests (fs_lora_add): out = base + scale B (A x) with the
// row's own A [rank][K] and B [N][rank].
#include "fs_internal.h"

namespace fsk {
namespace {

template <typename T>
__device__ __forceinline__ float val(const T* p, int64_t i) {
  if constexpr (sizeof(T) == 4) return p[i];
  else return __bfloat162float(p[i]);
}

constexpr int kT = 256;

// A block a row and part of the columns.
template <typename TX, typename TY>
__global__ void __launch_bounds__(kT) k_lora(const LoraArgs a) {
  __shared__ float low[128];
  const int row = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  const int which = a.adapter[row];
  const bool has = which >= 0 && which < a.n_adapters;
  if (has) {
    const TX* x = static_cast<const TX*>(a.x) + row * a.x_stride;
    for (int r = warp; r < a.rank; r += kT / 32) {
      const __nv_bfloat16* A = a.A + ((int64_t)which * a.rank + r) * a.K;
      float s = 0.0f;
      for (int k = lane; k < a.K; k += 32) s = fmaf(val(x, k), __bfloat162float(A[k]), s);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) low[r] = s * a.scale[which];
    }
  } else if (a.base == a.out) {
    return;
  }
  __syncthreads();
  const TY* base = static_cast<const TY*>(a.base) + row * a.base_stride;
  TY* out = static_cast<TY*>(a.out) + row * a.out_stride;
  for (int j = blockIdx.y * kT + tid; j < a.N; j += gridDim.y * kT) {
    float s = a.base ? val(base, j) : 0.0f;
    if (has) {
      float d = 0.0f;
      const __nv_bfloat16* B = a.B + ((int64_t)which * a.N + j) * a.rank;
      for (int r = 0; r < a.rank; ++r) d = fmaf(low[r], __bfloat162float(B[r]), d);
      s += d;
    }
    if constexpr (sizeof(TY) == 4) out[j] = s;
    else out[j] = __float2bfloat16_rn(s);
  }
}

}  // namespace

Launched launch_lora(const LoraArgs& a, int x_type, int y_type, int sms, cudaStream_t s) {
  const dim3 grid((unsigned)a.n, (unsigned)std::max(1, std::min((a.N + kT - 1) / kT, 4 * sms / a.n)));
  auto k = x_type == X_F32 ? (y_type == X_F32 ? k_lora<float, float> : k_lora<float, __nv_bfloat16>)
                           : (y_type == X_F32 ? k_lora<__nv_bfloat16, float>
                                              : k_lora<__nv_bfloat16, __nv_bfloat16>);
  Launched l;
  l.add(launch_k(k, grid, kT, 0, s, a));
  return l;
}

}  // namespace fsk
