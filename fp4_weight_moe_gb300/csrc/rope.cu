// Norms of queries and keys for each head, the rotation by their positions,
// and the store of keys and values into the cache of 4 bits
// (moe_fp4_qk_norm_rope).
//
// A head of D columns lies on D / 8 lanes, eight columns (16 bytes) each, so
// that a warp's loads and stores are whole rows; a warp takes up to kUnroll
// times as many heads of one token, all of one kind (queries, or keys with
// their values), with every load under way before the first sum.  The
// rotation's partner column i + rot / 2 is rot / 16 lanes away, a shuffle.
//
// Keys bound for the cache are computed in pairs of FP32 numbers (value and
// rest; sums and products without error by the published steps of D. E. Knuth,
// TAOCP 2, 4.2.2, and T. J. Dekker, "A floating-point technique for extending
// the available precision", 1971), good to about 2^-44: rounded to FP32 that
// is the number next to the formula's, whatever order sums are taken in, and
// so are its codes.  Straight FP32 is off by a unit or two, which moves about
// one code in 10^7 across a border of its rounding, by a third of its value.
#include "attention.cuh"
#include "fp8_quant.cuh"
#include "host.cuh"

namespace moe_fp4 {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kUnroll = 4;

// hi + lo, |lo| at most half a unit of hi.
struct Pair {
  float hi, lo;
};

__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fadd_rn(s, -a);
  return {s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -t)), __fadd_rn(b, -t))};
}
__device__ __forceinline__ Pair two_prod(float a, float b) {
  const float p = __fmul_rn(a, b);
  return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi);
  const float e = __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo));
  const float hi = __fadd_rn(s.hi, e);
  return {hi, __fadd_rn(e, -__fadd_rn(hi, -s.hi))};
}
__device__ __forceinline__ Pair operator*(Pair a, float b) {
  const Pair p = two_prod(a.hi, b);
  return {p.hi, __fmaf_rn(a.lo, b, p.lo)};
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  const Pair p = two_prod(a.hi, b.hi);
  return {p.hi, __fmaf_rn(a.hi, b.lo, __fmaf_rn(a.lo, b.hi, p.lo))};
}
__device__ __forceinline__ Pair lane_xor(Pair v, int o) {
  return {__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)};
}
__device__ __forceinline__ float lane_xor(float v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }

__device__ __forceinline__ void set(float& v, float x) { v = x; }
__device__ __forceinline__ void set(Pair& v, float x) { v = {x, 0.f}; }
__device__ __forceinline__ float value(Pair v) { return __fadd_rn(v.hi, v.lo); }

// 1 / sqrt(x): the hardware's approximation, and for a pair a step of
// y + y (r / 2 + 3 r^2 / 8) from the exact rest r = 1 - x y^2.
__device__ __forceinline__ float inverse_root(float x) { return rsqrtf(x); }
__device__ __forceinline__ Pair inverse_root(Pair x) {
  const float y = rsqrtf(x.hi);
  const Pair y2 = two_prod(y, y);
  float r = __fmaf_rn(-x.hi, y2.hi, 1.f);
  r = __fmaf_rn(-x.hi, y2.lo, r);
  r = __fmaf_rn(-x.lo, y2.hi, r);
  if (!(fabsf(r) < 1.f)) return {y, 0.f};  // (x zero or past FP32's ends)
  return {y, y * r * __fmaf_rn(0.375f, r, 0.5f)};
}

// A lane's factors of the rotation, the weights among them: column i becomes
// x_i own_i + partner_i other_i, times the norm.
struct Factors {
  float c[8], s[8], w[8], w_other[8];  // (s with its sign)
};

__device__ __forceinline__ float product(float a, float b, float) { return a * b; }
__device__ __forceinline__ Pair product(float a, float b, Pair) { return two_prod(a, b); }

__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
  const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(p[i] << 16);
    v[2 * i + 1] = __uint_as_float(p[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  uint32_t p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    p[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(p[0], p[1], p[2], p[3]);
}

// The rotation's partners of a lane's columns; zeros where nothing is turned.
// All lanes of the warp call it.
__device__ __forceinline__ uint4 partners(uint4 x, int from, bool turned, int interleaved) {
  uint4 o;
  if (interleaved) {
    o.x = __funnelshift_l(x.x, x.x, 16), o.y = __funnelshift_l(x.y, x.y, 16);
    o.z = __funnelshift_l(x.z, x.z, 16), o.w = __funnelshift_l(x.w, x.w, 16);
  } else {
    o.x = __shfl_sync(0xffffffffu, x.x, from), o.y = __shfl_sync(0xffffffffu, x.y, from);
    o.z = __shfl_sync(0xffffffffu, x.z, from), o.w = __shfl_sync(0xffffffffu, x.w, from);
  }
  return turned ? o : make_uint4(0, 0, 0, 0);
}

// A lane's eight columns of a head, normed and rotated.  F is float or Pair.
template <int D, class F>
__device__ __forceinline__ void norm_rotate(F (&y)[8], const float (&x)[8], const float (&o)[8], bool normed,
                                            const Factors& f, float eps) {
  F inv;
  if (normed) {
    F sum;
    set(sum, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = sum + product(x[i], x[i], sum);
#pragma unroll
    for (int n = D / 16; n > 0; n >>= 1) sum = sum + lane_xor(sum, n);
    F e;
    set(e, eps);
    inv = inverse_root(sum * (1.f / D) + e);
  } else {
    set(inv, 1.f);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    y[i] = (product(f.c[i], f.w[i], inv) * x[i] + product(f.s[i], f.w_other[i], inv) * o[i]) * inv;
}

// Eight of a block's sixteen columns (the others in lane ^ 1): their codes,
// and the block's scale byte.  `bad`: the block has an infinity or a NaN.
// Quotients are correctly rounded (quotients, fp8_quant.cuh), the scales' too.
__device__ __forceinline__ uint32_t quantise8(float (&u)[8], float scale, uint32_t& scale_byte, bool& bad) {
  if (scale != 1.f) {
#pragma unroll 1
    for (int i = 0; i < 8; ++i) {
      const float v = __fdiv_rn(u[0], scale);  // (around, so that the code is there once)
#pragma unroll
      for (int j = 0; j < 7; ++j) u[j] = u[j + 1];
      u[7] = v;
    }
  }
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(fabsf(u[i])));
  const float other = __shfl_xor_sync(0xffffffffu, top, 1);
  asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(other));
  bad = !(top < INFINITY);
  const float t = top * (1.f / 6.f);
  uint16_t s8;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %1;" : "=h"(s8) : "f"(fmaf(fmaf(t, -6.f, top), 1.f / 6.f, t)));
  scale_byte = s8 & 0xffu;
  const float s = e4m3_to_float(scale_byte);
  const float2 y = both(recip_rn(s)), neg = both(-s);
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 q = quotients(make_float2(u[2 * i], u[2 * i + 1]), neg, y);
    uint16_t b;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u16.u8 %0, t;\n\t}"
        : "=h"(b)
        : "f"(q.y), "f"(q.x));
    codes |= (uint32_t)(b & 0xffu) << (8 * i);
  }
  if (bad) scale_byte = 0x7fu;
  return bad || scale_byte == 0 ? 0 : codes;
}

// `per`: heads of a warp's task (a multiple of what it has under way at once).
template <int D>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(moe_fp4_qk_norm_rope_args a, int per_q, int q_tasks,
                                                                    int per_k, int tasks) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;  // heads side by side in a warp
  const int lane = threadIdx.x & 31, l = lane % kLanes, side = lane / kLanes;
  const int64_t task = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = task / tasks;
  if (t >= a.T) return;
  const int kind_task = (int)(task - t * tasks);
  const bool is_q = kind_task < q_tasks;
  const int first = is_q ? kind_task * per_q : (kind_task - q_tasks) * per_k;
  const int end = is_q ? min(first + per_q, a.Hq) : min(first + per_k, a.Hkv);
  const bool store = a.cache && !is_q;

  // weights and angles of this lane's columns
  Factors f;
  const int half = a.rot / 16;  // lanes of half the rotated columns
  const bool turned = a.rotary && 8 * l < a.rot, low = l < half;
  const int l_other = turned && !a.interleaved ? (low ? l + half : l - half) : l;
  const int from = lane - l + l_other;
  const void* wp = is_q ? a.w_q : a.w_k;
#pragma unroll
  for (int i = 0; i < 8; ++i) f.c[i] = 1.f, f.s[i] = 0.f, f.w[i] = 1.f, f.w_other[i] = 1.f;
  if (wp) {
    if (a.weights_f32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(wp));
      const float4 x0 = p[2 * l], x1 = p[2 * l + 1], o0 = p[2 * l_other], o1 = p[2 * l_other + 1];
      f.w[0] = x0.x, f.w[1] = x0.y, f.w[2] = x0.z, f.w[3] = x0.w;
      f.w[4] = x1.x, f.w[5] = x1.y, f.w[6] = x1.z, f.w[7] = x1.w;
      f.w_other[0] = o0.x, f.w_other[1] = o0.y, f.w_other[2] = o0.z, f.w_other[3] = o0.w;
      f.w_other[4] = o1.x, f.w_other[5] = o1.y, f.w_other[6] = o1.z, f.w_other[7] = o1.w;
    } else {
      unpack8(static_cast<const uint4*>(wp)[l], f.w);
      unpack8(static_cast<const uint4*>(wp)[l_other], f.w_other);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f.w[i] = a.offset + f.w[i], f.w_other[i] = a.offset + f.w_other[i];
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f.w_other[i] = f.w[i ^ 1];
    }
  }
  if (turned) {
    const int64_t pos = a.positions_i64 ? static_cast<const int64_t*>(a.positions)[t]
                                        : static_cast<const int32_t*>(a.positions)[t];
    if (pos < 0 || pos >= a.positions_max) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f.c[i] = f.s[i] = NAN;
    } else {
      const float* row = a.rotary + pos * a.rot;
      const float4* c = reinterpret_cast<const float4*>(row + (a.interleaved ? 4 * l : low ? 8 * l : 8 * (l - half)));
      const float4* s = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(c) + a.rot / 2);
      const float4 c0 = c[0], s0 = s[0];
      if (a.interleaved) {
        f.c[0] = f.c[1] = c0.x, f.c[2] = f.c[3] = c0.y, f.c[4] = f.c[5] = c0.z, f.c[6] = f.c[7] = c0.w;
        f.s[1] = s0.x, f.s[3] = s0.y, f.s[5] = s0.z, f.s[7] = s0.w;
        f.s[0] = -s0.x, f.s[2] = -s0.y, f.s[4] = -s0.z, f.s[6] = -s0.w;
      } else {
        const float4 c1 = c[1], s1 = s[1];
        f.c[0] = c0.x, f.c[1] = c0.y, f.c[2] = c0.z, f.c[3] = c0.w;
        f.c[4] = c1.x, f.c[5] = c1.y, f.c[6] = c1.z, f.c[7] = c1.w;
        f.s[0] = s0.x, f.s[1] = s0.y, f.s[2] = s0.z, f.s[3] = s0.w;
        f.s[4] = s1.x, f.s[5] = s1.y, f.s[6] = s1.z, f.s[7] = s1.w;
        if (low) {
#pragma unroll
          for (int i = 0; i < 8; ++i) f.s[i] = -f.s[i];
        }
      }
    }
  }

  const __nv_bfloat16* in = static_cast<const __nv_bfloat16*>(is_q ? a.q_in : a.k_in) +
                            t * (is_q ? a.q_row : a.k_row) + 8 * l;
  const int64_t step = is_q ? a.q_head : a.k_head;
  if (!store) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      f.c[i] *= f.w[i], f.s[i] *= f.w_other[i];
      f.w[i] = f.w_other[i] = 1.f;
    }
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(is_q ? a.q_out : a.k_out) +
                         t * (is_q ? a.q_out_row : a.k_out_row) + 8 * l;
    const int64_t out_step = is_q ? a.q_out_head : a.k_out_head;
#pragma unroll 1
    for (int base = first; base < end; base += kUnroll * kHeads) {
      uint4 raw[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = base + u * kHeads + side;
        raw[u] = h < end ? *reinterpret_cast<const uint4*>(in + h * step) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (base + u * kHeads >= end) break;  // (the same for the whole warp)
        float x[8], o[8], y[8];
        unpack8(raw[u], x);
        unpack8(partners(raw[u], from, turned, a.interleaved), o);
        norm_rotate<D>(y, x, o, wp != nullptr, f, a.eps);
        const int h = base + u * kHeads + side;
        if (h < end) *reinterpret_cast<uint4*>(out + h * out_step) = pack8(y);
      }
    }
    return;
  }

  const int64_t slot = a.slots[t];
  const bool kept = slot >= 0 && slot < (int64_t)a.pages * a.page_size;
  const __nv_bfloat16* vin = static_cast<const __nv_bfloat16*>(a.v_in) + t * a.v_row + 8 * l;
#pragma unroll 1
  for (int base = first; base < end; base += kHeads) {
    const int h = base + side;
    const uint4 raw = h < end ? *reinterpret_cast<const uint4*>(in + h * step) : make_uint4(0, 0, 0, 0);
    const uint4 vals = h < end ? *reinterpret_cast<const uint4*>(vin + h * a.v_head) : make_uint4(0, 0, 0, 0);
    float x[8], o[8], u[8];
    Pair p[8];
    unpack8(raw, x);
    unpack8(partners(raw, from, turned, a.interleaved), o);
    norm_rotate<D>(p, x, o, wp != nullptr, f, a.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = value(p[i]);
    uint32_t k_scale, v_scale;
    bool k_bad, v_bad;
    const uint32_t k_codes = quantise8(u, a.k_scale, k_scale, k_bad);
    unpack8(vals, u);
    const uint32_t v_codes = quantise8(u, a.v_scale, v_scale, v_bad);
    const unsigned bad = __ballot_sync(0xffffffffu, k_bad || v_bad) >> (side * kLanes);
    if ((kLanes == 32 ? bad : bad & ((1u << (kLanes % 32)) - 1)) != 0) k_scale = 0x7fu;
    if (h < end && kept) {
      const CachePlace at = cache_place(slot, h, a.Hkv, a.page_size, D);
      uint8_t* k = static_cast<uint8_t*>(a.cache);
      uint8_t* v = k + cache_half_bytes(D);
      *reinterpret_cast<uint32_t*>(k + at.codes + 4 * l) = k_codes;
      *reinterpret_cast<uint32_t*>(v + at.codes + 4 * l) = v_codes;
      if (l % 2 == 0) {
        k[at.scales + l / 2] = (uint8_t)k_scale;
        v[at.scales + l / 2] = (uint8_t)v_scale;
      }
    }
  }
}

template <int D>
cudaError_t launch_dim(const moe_fp4_qk_norm_rope_args& a, cudaStream_t st) {
  constexpr int kHeads = 32 / (D / 8), kAtOnce = kUnroll * kHeads;
  int sms = 0;
  const cudaError_t e = current_device_sms(&sms);
  if (e != cudaSuccess) return e;
  // few tokens: a task of what a warp has under way; many: all of a token's
  // queries, so that its weights and angles are read once
  const bool many = a.T >= 16 * sms;
  const int per_q = many ? ceil_div(a.Hq, kAtOnce) * kAtOnce : kAtOnce;
  const int per_k = !a.cache ? per_q : many ? 4 * kHeads : kHeads;
  const int q_tasks = ceil_div(a.Hq, per_q), tasks = q_tasks + ceil_div(a.Hkv, per_k);
  const int64_t grid = ((int64_t)a.T * tasks + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_dependent(qk_norm_rope_kernel<D>, (unsigned)grid, kRopeThreads, st, a, per_q, q_tasks, per_k, tasks);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const moe_fp4_qk_norm_rope_args& a, cudaStream_t st) {
  switch (a.D) {
    case 64: return launch_dim<64>(a, st);
    case 128: return launch_dim<128>(a, st);
    default: return launch_dim<256>(a, st);
  }
}

}  // namespace moe_fp4
