// FP8 (E4M3) activations with a scale per 128 columns: the pieces shared by
// the quantiser, the product kernel that quantises its own tokens, and the
// norm that hands its output on in FP8.  A block's 128 values lie eight per
// lane on 16 consecutive lanes.
#pragma once

#include "common.cuh"

namespace moe_fp4 {

__device__ __forceinline__ void bf16x8_to_float(uint4 u, float (&v)[8]) {
  const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(p[i] << 16);
    v[2 * i + 1] = __uint_as_float(p[i] & 0xffff0000u);
  }
}

// Largest magnitude of a block (16 lanes); NaNs are passed over.
__device__ __forceinline__ float block_amax(const float (&v)[8]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = fmaxf(a, fabsf(v[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

// The block's scale: amax / 448, or 1 where that is zero (an all-zero block,
// or one below FP32's reach).
__device__ __forceinline__ float block_scale(float amax) {
  const float s = __fdiv_rn(amax, 448.f);
  return s == 0.f ? 1.f : s;
}

// Eight E4M3 bytes of v / s, the quotients correctly rounded to FP32 before
// they are rounded to E4M3 (to nearest even, saturating).  Away from FP32's
// ends the quotients come from the correctly rounded reciprocal y of s: q =
// v y is within two units, and q + (v - q s) y, both steps fused, is the
// correctly rounded quotient (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990): three operations
// a value, where the quantiser would spend more on divisions than on its
// memory traffic.  Quotients too small for the exact remainder are far below
// half of E4M3's least value and round to zero either way.
__device__ __forceinline__ uint2 e4m3_quotients(const float (&v)[8], float s) {
  float q[8];
  if (s > 0x1p-60f && s < 0x1p60f) {
    const float y = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = v[i] * y;
      q[i] = fmaf(fmaf(-t, s, v[i]), y, t);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(v[i], s);
  }
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(q[4 * i + 1]), "f"(q[4 * i]));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(q[4 * i + 3]), "f"(q[4 * i + 2]));
    w[i] = (uint32_t)lo | ((uint32_t)hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

}  // namespace moe_fp4
