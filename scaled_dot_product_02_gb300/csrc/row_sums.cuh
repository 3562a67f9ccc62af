// row_sums.cuh -- a warp's maxima and sums over its lanes, for the kernels that
// have a key a thread and a query row a register.
#pragma once
#include <cstdint>

namespace sdpa {

__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Sum v[n] over the 32 lanes, leaving N/32 sums (or one, twice) a lane: rows
// N <= 32: lane / (32 / N), N = 64: 2 * lane + i.
template <int N>
__device__ __forceinline__ void scatter_sum(float (&v)[N], int lane) {
  int o = 16;
#pragma unroll
  for (int cnt = N; cnt > 1 && o >= 1; cnt /= 2, o /= 2) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < cnt / 2; ++i) {
      const float send = up ? v[i] : v[i + cnt / 2];
      const float keep = up ? v[i + cnt / 2] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
#pragma unroll
  for (int x = 16 / N; x >= 1; x /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], x);
}

}  // namespace sdpa
