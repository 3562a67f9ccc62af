// row_pass.cuh -- the softmax pass over one row of scores in TMEM, shared by the
// head_dim 128 forward (fwd.cu) and the paged-cache attention (paged_pair.cu).
#pragma once
#include "common.cuh"
#include "ptx.cuh"

namespace sdpa {

// One pass of the head_dim 128 softmax over the 128 scores of a row held in
// TMEM: t = S*scale*log2e - mb, P = exp2(t) packed to 16-bit pairs (zero
// where masked), the row sum of P and the largest t among allowed keys.
template <bool MASK, class E>
__device__ __forceinline__ void p_pass(uint32_t scol, float sl2, float mb, int kb, int lo, int hi,
                                       uint32_t (&pk)[64], float& rs, float& tmax) {
  const float2 sc = make_float2(sl2, sl2), nm = make_float2(-mb, -mb);
  float2 acc = make_float2(0.f, 0.f);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t u[32];
    float cmax = 0.f;
    if (MASK)
      tmem_ld32(scol + c * 32, u);
    else
      tmem_ld32_max(scol + c * 32, u, cmax);
    tmem_wait_ld();
    reg_fence(u);
    if (!MASK) {
      // the load returned the chunk's max score; the rounding of the exponent
      // being monotone, fma(max, scale*log2e, -mb) is the chunk's largest one
      asm volatile("" : "+f"(cmax));
      tmax = fmaxf(tmax, __fmaf_rn(cmax, sl2, -mb));
    }
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      float2 t = ffma2(make_float2(__uint_as_float(u[e]), __uint_as_float(u[e + 1])), sc, nm);
      if (MASK) {
        const int key = kb + c * 32 + e;
        t.x = in_range(key, lo, hi) ? t.x : -INFINITY;
        t.y = in_range(key + 1, lo, hi) ? t.y : -INFINITY;
        tmax = fmaxf(tmax, fmaxf(t.x, t.y));
      }
      const float2 p = make_float2(ex2(t.x), ex2(t.y));
      pk[c * 16 + e / 2] = E::pack(p.x, p.y);
      acc = fadd2(acc, p);
    }
  }
  rs = acc.x + acc.y;
}

}  // namespace sdpa
