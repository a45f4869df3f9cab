// FP8 (E4M3) activations with a scale per 128 columns: the pieces shared by
// the quantiser, the product kernel that quantises its own tokens, and the
// norm that hands its output on in FP8 (the reciprocal by the router, too).  A
// block's 128 values lie V per lane (8 or 16) on 128 / V consecutive lanes.
#pragma once

#include "common.cuh"

namespace moe_fp4 {

__device__ __forceinline__ void bf16x8_to_float(uint4 u, float* v) {
  const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(p[i] << 16);
    v[2 * i + 1] = __uint_as_float(p[i] & 0xffff0000u);
  }
}

// Largest magnitude of a block; NaNs are passed over.
template <int V>
__device__ __forceinline__ float block_amax(const float (&v)[V]) {
  float a = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) a = fmaxf(a, fabsf(v[i]));
#pragma unroll
  for (int o = 64 / V; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
  return a;
}

// Quotients without branches, and two at a time, from a reciprocal y of the
// divisor s: q + (v - q s) y, both steps fused, is the correctly rounded
// quotient where q is within a unit of it and y is the correctly rounded
// reciprocal (P. Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990): three operations a value, where the
// kernels here would spend more on divisions than on their memory traffic.
// q = v y itself may be off by up to a unit and a half, exclusive (v times
// the half unit of y, and its own half), but the last step can only go wrong
// for quotients next to a midpoint of two values, which are half a unit or a
// unit and a half from q, and the latter is out of reach.  Away from FP32's
// ends only; a zero may lose its sign.
__device__ __forceinline__ float2 quotients(float2 v, float2 s_neg, float2 y) {
  const float2 t = fmul2(v, y);
  return ffma2(ffma2(t, s_neg, v), y, t);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// 1 / x, 2^-126 < x < 2^126, correctly rounded, without branches: a step of y
// + y (1 - x y) on the hardware's approximation, which is within a unit (same
// source; compared with the IEEE reciprocal for all 2^23 significands).
__device__ __forceinline__ float recip_rn(float x) {
  float y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return fmaf(y, fmaf(-x, y, 1.0f), y);
}

// The same of -s_neg, two at a time.
__device__ __forceinline__ float2 reciprocals(float2 s_neg) {
  float2 y;
  asm("rcp.approx.f32 %0, %1;" : "=f"(y.x) : "f"(-s_neg.x));
  asm("rcp.approx.f32 %0, %1;" : "=f"(y.y) : "f"(-s_neg.y));
  return ffma2(y, ffma2(s_neg, y, both(1.f)), y);
}

// The block's scale: amax / 448, or 1 where that is zero (an all-zero block,
// or one below FP32's reach).
__device__ __forceinline__ float block_scale(float amax) {
  if (amax > 0x1p-60f && amax < 0x1p60f) {
    const float y = 1.f / 448.f, t = amax * y;
    return fmaf(fmaf(t, -448.f, amax), y, t);
  }
  const float s = __fdiv_rn(amax, 448.f);
  return s == 0.f ? 1.f : s;
}

// E4M3 bytes of v / s, the quotients correctly rounded to FP32 before they
// are rounded to E4M3 (to nearest even, saturating).  Quotients too small for
// the exact remainder are far below half of E4M3's least value and round to
// zero either way.
template <int V>
__device__ __forceinline__ void e4m3_quotients(const float (&v)[V], float s, uint32_t (&w)[V / 4]) {
  float2 q[V / 2];
  if (s > 0x1p-70f && s < 0x1p60f) {
    const float2 y = both(reciprocals(both(-s)).x);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) q[i] = quotients(make_float2(v[2 * i], v[2 * i + 1]), both(-s), y);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) q[i] = make_float2(__fdiv_rn(v[2 * i], s), __fdiv_rn(v[2 * i + 1], s));
  }
#pragma unroll
  for (int i = 0; i < V / 4; ++i) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(q[2 * i].y), "f"(q[2 * i].x));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(q[2 * i + 1].y), "f"(q[2 * i + 1].x));
    w[i] = (uint32_t)lo | ((uint32_t)hi << 16);
  }
}

__device__ __forceinline__ uint2 e4m3_quotients(const float (&v)[8], float s) {
  uint32_t w[2];
  e4m3_quotients(v, s, w);
  return make_uint2(w[0], w[1]);
}

}  // namespace moe_fp4
