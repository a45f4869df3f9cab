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
__device__ __forceinline__ Pair operator-(Pair a) { return {-a.hi, -a.lo}; }
__device__ __forceinline__ Pair lane_xor(Pair v, int o) {
  return {__shfl_xor_sync(0xffffffffu, v.hi, o), __shfl_xor_sync(0xffffffffu, v.lo, o)};
}
__device__ __forceinline__ float lane_xor(float v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }
__device__ __forceinline__ Pair lane_from(Pair v, int l) {
  return {__shfl_sync(0xffffffffu, v.hi, l), __shfl_sync(0xffffffffu, v.lo, l)};
}
__device__ __forceinline__ float lane_from(float v, int l) { return __shfl_sync(0xffffffffu, v, l); }

__device__ __forceinline__ void set(float& v, float x) { v = x; }
__device__ __forceinline__ void set(Pair& v, float x) { v = {x, 0.f}; }
__device__ __forceinline__ float value(float v) { return v; }
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

struct Angles {
  float c[8], s[8];  // halves: of the lane's eight columns; interleaved: of its four pairs
};

// A lane's eight columns of a head, normed and rotated.  F is float or Pair.
template <int D, class F>
__device__ __forceinline__ void norm_rotate(F (&y)[8], const float (&x)[8], const float (&w)[8], bool normed,
                                            const Angles& g, const moe_fp4_qk_norm_rope_args& a, int l, int lane) {
  constexpr int kLanes = D / 8;
  F inv;
  if (normed) {
    F sum;
    set(sum, 0.f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      F v;
      set(v, x[i]);
      sum = sum + v * x[i];
    }
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) sum = sum + lane_xor(sum, o);
    F e;
    set(e, a.eps);
    inv = inverse_root(sum * (1.f / D) + e);
  } else {
    set(inv, 1.f);
  }
  F v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    set(v[i], x[i]);
    v[i] = v[i] * w[i];
  }
  if (a.rotary) {
    if (a.interleaved) {
      if (8 * l < a.rot) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const F p = v[2 * i], q = v[2 * i + 1];
          v[2 * i] = p * g.c[i] + -(q * g.s[i]);
          v[2 * i + 1] = q * g.c[i] + p * g.s[i];
        }
      }
    } else {
      const int half = a.rot / 16;  // lanes
      const bool first = l < half;
      const int from = lane + (l < 2 * half ? (first ? half : -half) : 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const F other = lane_from(v[i], from);
        const F turned = v[i] * g.c[i] + (first ? -(other * g.s[i]) : other * g.s[i]);
        if (l < 2 * half) v[i] = turned;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = v[i] * inv;
}

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

// Eight of a block's sixteen columns (the others in lane ^ 1): their codes,
// and the block's scale byte.  `bad`: the block has an infinity or a NaN.
__device__ __forceinline__ uint32_t quantise8(const float (&v)[8], float scale, uint32_t& scale_byte, bool& bad) {
  float u[8], top = 0.f;
  bool fine = true;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    u[i] = scale == 1.f ? v[i] : __fdiv_rn(v[i], scale);
    top = fmaxf(top, fabsf(u[i]));
    fine = fine && fabsf(u[i]) < INFINITY;
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  bad = !fine;
  bad = __shfl_xor_sync(0xffffffffu, bad, 1) || bad;
  uint16_t s8;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %1;" : "=h"(s8) : "f"(__fdiv_rn(top, 6.f)));
  scale_byte = s8 & 0xffu;
  const float s = e4m3_to_float(scale_byte);
  uint32_t codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = s > 0.f ? __fdiv_rn(u[2 * i], s) : 0.f, hi = s > 0.f ? __fdiv_rn(u[2 * i + 1], s) : 0.f;
    uint16_t b;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u16.u8 %0, t;\n\t}"
        : "=h"(b)
        : "f"(hi), "f"(lo));
    codes |= (uint32_t)(b & 0xffu) << (8 * i);
  }
  if (bad) {
    scale_byte = 0x7fu;
    codes = 0;
  }
  return codes;
}

template <int D>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(moe_fp4_qk_norm_rope_args a, int q_tasks,
                                                                    int tasks) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;  // heads side by side in a warp
  const int lane = threadIdx.x & 31, l = lane % kLanes, side = lane / kLanes;
  const int64_t task = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = task / tasks;
  if (t >= a.T) return;
  const int kind_task = (int)(task % tasks);
  const bool is_q = kind_task < q_tasks;
  const int heads = is_q ? a.Hq : a.Hkv;
  const int first = (is_q ? kind_task : kind_task - q_tasks) * kUnroll * kHeads + side;
  const bool store = a.cache && !is_q;

  const __nv_bfloat16* in = static_cast<const __nv_bfloat16*>(is_q ? a.q_in : a.k_in) +
                            t * (is_q ? a.q_row : a.k_row) + 8 * l;
  const int64_t step = is_q ? a.q_head : a.k_head;
  uint4 raw[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int h = first + u * kHeads;
    raw[u] = h < heads ? *reinterpret_cast<const uint4*>(in + h * step) : make_uint4(0, 0, 0, 0);
  }
  uint4 vals[kUnroll];
  int64_t slot = -1;
  if (store) {
    slot = a.slots[t];
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v_in) + t * a.v_row + 8 * l;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = first + u * kHeads;
      vals[u] = h < heads ? *reinterpret_cast<const uint4*>(v + h * a.v_head) : make_uint4(0, 0, 0, 0);
    }
  }

  float w[8];
  const void* wp = is_q ? a.w_q : a.w_k;
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.f;
  if (wp) {
    if (a.weights_f32) {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(wp) + 8 * l);
      const float4 lo = p[0], hi = p[1];
      w[0] = lo.x, w[1] = lo.y, w[2] = lo.z, w[3] = lo.w, w[4] = hi.x, w[5] = hi.y, w[6] = hi.z, w[7] = hi.w;
    } else {
      unpack8(*reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(wp) + 8 * l), w);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = a.offset + w[i];
  }

  Angles g;
#pragma unroll
  for (int i = 0; i < 8; ++i) g.c[i] = 1.f, g.s[i] = 0.f;
  if (a.rotary && 8 * l < a.rot) {
    const int64_t pos = a.positions_i64 ? static_cast<const int64_t*>(a.positions)[t]
                                        : static_cast<const int32_t*>(a.positions)[t];
    if (pos < 0 || pos >= a.positions_max) {
#pragma unroll
      for (int i = 0; i < 8; ++i) g.c[i] = g.s[i] = NAN;
    } else {
      const float* row = a.rotary + pos * a.rot;
      const int half = a.rot / 2, at = a.interleaved ? 4 * l : 8 * l < half ? 8 * l : 8 * l - half;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (i == 1 && a.interleaved) break;
        const float4 c = *reinterpret_cast<const float4*>(row + at + 4 * i);
        const float4 s = *reinterpret_cast<const float4*>(row + half + at + 4 * i);
        g.c[4 * i] = c.x, g.c[4 * i + 1] = c.y, g.c[4 * i + 2] = c.z, g.c[4 * i + 3] = c.w;
        g.s[4 * i] = s.x, g.s[4 * i + 1] = s.y, g.s[4 * i + 2] = s.z, g.s[4 * i + 3] = s.w;
      }
    }
  }

  if (!store) {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(is_q ? a.q_out : a.k_out) +
                         t * (is_q ? a.q_out_row : a.k_out_row) + 8 * l;
    const int64_t out_step = is_q ? a.q_out_head : a.k_out_head;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (first - side + u * kHeads >= heads) break;  // (the same for the whole warp)
      float x[8], y[8];
      unpack8(raw[u], x);
      norm_rotate<D>(y, x, w, wp != nullptr, g, a, l, lane);
      const int h = first + u * kHeads;
      if (h < heads) *reinterpret_cast<uint4*>(out + h * out_step) = pack8(y);
    }
    return;
  }

  const bool kept = slot >= 0 && slot < (int64_t)a.pages * a.page_size;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (first - side + u * kHeads >= heads) break;
    const int h = first + u * kHeads;
    float x[8], y[8];
    Pair p[8];
    unpack8(raw[u], x);
    norm_rotate<D>(p, x, w, wp != nullptr, g, a, l, lane);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = value(p[i]);
    uint32_t k_scale, v_scale;
    bool k_bad, v_bad;
    const uint32_t k_codes = quantise8(y, a.k_scale, k_scale, k_bad);
    unpack8(vals[u], x);
    const uint32_t v_codes = quantise8(x, a.v_scale, v_scale, v_bad);
    const unsigned bad = __ballot_sync(0xffffffffu, k_bad || v_bad) >> (side * kLanes);
    if ((kLanes == 32 ? bad : bad & ((1u << (kLanes % 32)) - 1)) != 0) k_scale = 0x7fu;
    if (h < heads && kept) {
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
  const int per = kUnroll * 32 / (D / 8);
  const int q_tasks = ceil_div(a.Hq, per), tasks = q_tasks + ceil_div(a.Hkv, per);
  const int64_t grid = ((int64_t)a.T * tasks + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_dependent(qk_norm_rope_kernel<D>, (unsigned)grid, kRopeThreads, st, a, q_tasks, tasks);
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
