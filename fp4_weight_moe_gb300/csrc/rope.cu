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
// Keys bound for the cache have to give the codes of the FP32 number next to
// the formula's, whatever order sums are taken in; straight FP32 is off by a
// few units, which moves about one code in 10^7 across a border of its
// rounding, by a third of its value.  So each key is quantised from FP32 with
// its bound of error added and taken away: where both give the same scales and
// codes (all but one head in a hundred) they are the right ones.  The others,
// and all keys without a norm, whose size that bound does not know, are
// computed again in pairs of FP32 numbers (value and rest; sums and
// products without error by the published steps of D. E. Knuth, TAOCP 2,
// 4.2.2, and T. J. Dekker, "A floating-point technique for extending the
// available precision", 1971), good to about 2^-44.
//
// 8192 tokens of 32 query and 8 key heads of 128 columns (178 MB): 46 us, 3.9
// TB/s; bound by issue (69% of the slots, the ALU 59% busy: a quotient, two
// borders and a code for each of the cached values), not by memory (without
// the cache 1001 tokens of wide heads take 7.2 us, which is 2.6 TB/s of L2).
// The same with keys that have no norm, each computed twice: 58 us.
#include "attention.cuh"
#include "fp8_quant.cuh"
#include "host.cuh"

namespace moe_fp4 {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kUnroll = 2;

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
// 1 / sqrt(x): the hardware's approximation, and for a pair a step of
// y + y (r / 2 + 3 r^2 / 8) from the exact rest r = 1 - x y^2.
__device__ __forceinline__ Pair inverse_root(Pair x) {
  const float y = rsqrtf(x.hi);
  const Pair y2 = two_prod(y, y);
  float r = __fmaf_rn(-x.hi, y2.hi, 1.f);
  r = __fmaf_rn(-x.hi, y2.lo, r);
  r = __fmaf_rn(-x.lo, y2.hi, r);
  if (!(fabsf(r) < 1.f)) return {y, 0.f};  // (x zero or past FP32's ends)
  return {y, y * r * __fmaf_rn(0.375f, r, 0.5f)};
}

// The weights of a lane's columns and of their partners', and the angles of a
// position (halves: eight; interleaved: four pairs').
struct Weights {
  float own[8], other[8];
};
struct Angles {
  float4 c[2], s[2];
};

__device__ __forceinline__ void unpack8(uint4 u, float (&v)[8]) {
  const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(p[i] << 16);
    v[2 * i + 1] = __uint_as_float(p[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint32_t pack2(float2 v) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// A lane's part in a head: its place, and the lane of the rotation's partners.
struct Lane {
  int l, half, l_other, from;
  bool turned, low;
};
template <int D>
__device__ __forceinline__ Lane lane_of(const moe_fp4_qk_norm_rope_args& a, int lane) {
  Lane at;
  at.l = lane % (D / 8);
  at.half = a.rot / 16;  // lanes of half the rotated columns
  at.turned = a.rotary && 8 * at.l < a.rot;
  at.low = at.l < at.half;
  at.l_other = at.turned && !a.interleaved ? (at.low ? at.l + at.half : at.l - at.half) : at.l;
  at.from = lane - at.l + at.l_other;
  return at;
}

__device__ __forceinline__ void load_weights(Weights& w, const moe_fp4_qk_norm_rope_args& a, const void* wp,
                                             const Lane& at) {
#pragma unroll
  for (int i = 0; i < 8; ++i) w.own[i] = w.other[i] = 1.f;
  if (!wp) return;
  if (a.weights_f32) {
    const float4* p = static_cast<const float4*>(wp);
    const float4 x0 = p[2 * at.l], x1 = p[2 * at.l + 1], o0 = p[2 * at.l_other], o1 = p[2 * at.l_other + 1];
    w.own[0] = x0.x, w.own[1] = x0.y, w.own[2] = x0.z, w.own[3] = x0.w;
    w.own[4] = x1.x, w.own[5] = x1.y, w.own[6] = x1.z, w.own[7] = x1.w;
    w.other[0] = o0.x, w.other[1] = o0.y, w.other[2] = o0.z, w.other[3] = o0.w;
    w.other[4] = o1.x, w.other[5] = o1.y, w.other[6] = o1.z, w.other[7] = o1.w;
  } else {
    unpack8(static_cast<const uint4*>(wp)[at.l], w.own);
    unpack8(static_cast<const uint4*>(wp)[at.l_other], w.other);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) w.own[i] = a.offset + w.own[i], w.other[i] = a.offset + w.other[i];
  if (a.interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w.other[i] = w.own[i ^ 1];
  }
}

__device__ __forceinline__ int64_t position(const moe_fp4_qk_norm_rope_args& a, int64_t t) {
  if (!a.rotary) return 0;
  return a.positions_i64 ? static_cast<const int64_t*>(a.positions)[t] : static_cast<const int32_t*>(a.positions)[t];
}

__device__ __forceinline__ void load_angles(Angles& g, const moe_fp4_qk_norm_rope_args& a, int64_t pos, const Lane& at) {
  const float none = pos < 0 || pos >= a.positions_max ? NAN : 1.f;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    g.c[i] = make_float4(none, none, none, none), g.s[i] = make_float4(none, none, none, none);
  if (!at.turned || none != 1.f) return;
  const float* row = a.rotary + pos * a.rot;
  const float4* c = reinterpret_cast<const float4*>(row + (a.interleaved ? 4 * at.l : at.low ? 8 * at.l : 8 * (at.l - at.half)));
  const float4* s = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(c) + a.rot / 2);
  g.c[0] = c[0], g.s[0] = s[0];
  if (!a.interleaved) g.c[1] = c[1], g.s[1] = s[1];
}

// Column i becomes x_i c_i + partner_i s_i, times the norm: cosines, and sines
// with their signs, for each of the lane's columns.
__device__ __forceinline__ void spread_angles(float (&c)[8], float (&s)[8], const Angles& g, const Lane& at,
                                              int interleaved) {
  if (!at.turned) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
    return;
  }
  const float c0[4] = {g.c[0].x, g.c[0].y, g.c[0].z, g.c[0].w}, c1[4] = {g.c[1].x, g.c[1].y, g.c[1].z, g.c[1].w};
  const float s0[4] = {g.s[0].x, g.s[0].y, g.s[0].z, g.s[0].w}, s1[4] = {g.s[1].x, g.s[1].y, g.s[1].z, g.s[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float ch = i < 4 ? c0[i % 4] : c1[i % 4], sh = i < 4 ? s0[i % 4] : s1[i % 4];
    c[i] = interleaved ? c0[i / 2] : ch;
    s[i] = interleaved ? (i % 2 ? s0[i / 2] : -s0[i / 2]) : at.low ? -sh : sh;
  }
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

// A lane's eight columns of a key, normed and rotated in pairs, as FP32.
template <int D>
__device__ __forceinline__ void norm_rotate_pairs(float2 (&y)[4], const moe_fp4_qk_norm_rope_args& a, int64_t t, uint4 raw,
                                                  uint4 partner, const Lane& at) {
  Weights w;
  load_weights(w, a, a.w_k, at);
  Angles g;
  load_angles(g, a, position(a, t), at);
  float c[8], s[8], x[8], o[8];
  spread_angles(c, s, g, at, a.interleaved);
  unpack8(raw, x);
  unpack8(partner, o);
  Pair inv = {1.f, 0.f};
  if (a.w_k) {
    Pair sum = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = sum + two_prod(x[i], x[i]);
#pragma unroll
    for (int n = D / 16; n > 0; n >>= 1) sum = sum + lane_xor(sum, n);
    inv = inverse_root(sum * (1.f / D) + Pair{a.eps, 0.f});
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const Pair v = (two_prod(c[i], w.own[i]) * x[i] + two_prod(s[i], w.other[i]) * o[i]) * inv;
    x[i] = __fadd_rn(v.hi, v.lo);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = make_float2(x[2 * i], x[2 * i + 1]);
}

// The same in FP32, two columns at a time, with factors that have the weights.
template <int D>
__device__ __forceinline__ void norm_rotate(float2 (&y)[4], uint4 raw, uint4 partner, bool normed, const float2 (&c)[4],
                                            const float2 (&s)[4], float eps) {
  float xs[8], os[8];
  unpack8(raw, xs);
  unpack8(partner, os);
  float2 x[4], o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = make_float2(xs[2 * i], xs[2 * i + 1]), o[i] = make_float2(os[2 * i], os[2 * i + 1]);
  float inv = 1.f;
  if (normed) {
    float2 sum = fmul2(x[0], x[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) sum = ffma2(x[i], x[i], sum);
    float all = sum.x + sum.y;
#pragma unroll
    for (int n = D / 16; n > 0; n >>= 1) all += __shfl_xor_sync(0xffffffffu, all, n);
    inv = rsqrtf(fmaf(all, 1.f / D, eps));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = fmul2(ffma2(x[i], c[i], fmul2(o[i], s[i])), both(inv));
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ uint32_t e4m3_bits(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %1;" : "=h"(r) : "f"(v));
  return r & 0xffu;
}

__device__ __forceinline__ uint32_t e2m1_pair(float2 q) {
  uint16_t b;
  asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\tcvt.u16.u8 %0, t;\n\t}" : "=h"(b) : "f"(q.y), "f"(q.x));
  return b & 0xffu;
}

// top / 6, correctly rounded (quotients, fp8_quant.cuh).
__device__ __forceinline__ float sixth(float top) {
  const float t = top * (1.f / 6.f);
  return fmaf(fmaf(t, -6.f, top), 1.f / 6.f, t);
}

// Eight of a block's sixteen columns (the others in lane ^ 1): their codes,
// and the block's scale byte.  `bad`: the block has an infinity or a NaN.
// kBounded: the columns are off by up to `off`; false where that leaves their
// codes or scale open.
struct Quantised {
  uint32_t codes, scale;
  bool bad;
};
template <bool kBounded>
__device__ __forceinline__ bool quantise8(const float2 (&u)[4], float off, Quantised& r) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max_nan(max_nan(top, fabsf(u[i].x)), fabsf(u[i].y));
  top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
  r.bad = !(top < INFINITY);
  r.scale = e4m3_bits(sixth(kBounded ? top + off : top));
  bool sure = !kBounded || r.scale == e4m3_bits(sixth(top - off));
  const float s = e4m3_to_float(r.scale), y = recip_rn(s);
  r.codes = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kBounded) {
      const float2 q = fmul2(u[i], both(y)), e = both(off * y);
      const uint32_t up = e2m1_pair(make_float2(q.x + e.x, q.y + e.y)), down = e2m1_pair(make_float2(q.x - e.x, q.y - e.y));
      sure = sure && up == down;
      r.codes |= up << (8 * i);
    } else {
      r.codes |= e2m1_pair(quotients(u[i], both(-s), both(y))) << (8 * i);
    }
  }
  if (r.bad || r.scale == 0) r.codes = 0;
  if (r.bad) r.scale = 0x7fu;
  return sure || r.bad;
}

__device__ __forceinline__ void divide8(float2 (&u)[4], float scale) {
  if (scale == 1.f) return;
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {  // (around, so that the code is there once)
    const float2 v = make_float2(__fdiv_rn(u[0].x, scale), __fdiv_rn(u[0].y, scale));
    u[0] = u[1], u[1] = u[2], u[2] = u[3], u[3] = v;
  }
}

// Whether `v` holds on any lane of this lane's head.
template <int D>
__device__ __forceinline__ bool head_any(bool v, int side) {
  constexpr int kLanes = D / 8;
  const unsigned lanes = __ballot_sync(0xffffffffu, v) >> (side * kLanes);
  return (kLanes == 32 ? lanes : lanes & ((1u << (kLanes % 32)) - 1)) != 0;
}

// A warp's task: per_q queries or per_k keys of a token.  Its loads are one
// iteration ahead.  (Several tokens to a task, with the weights kept, needed
// more registers than there are: 77 us where this took 49.)
template <int D, int kBlocks = 7>
__global__ void __launch_bounds__(kRopeThreads, kBlocks) qk_norm_rope_kernel(moe_fp4_qk_norm_rope_args a, int per_q,
                                                                             int q_tasks, int per_k, int tasks) {
  constexpr int kLanes = D / 8, kHeads = 32 / kLanes;  // heads side by side in a warp
  const int lane = threadIdx.x & 31, side = lane / kLanes;
  const int64_t task = ((int64_t)blockIdx.x * kRopeThreads + threadIdx.x) >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = task / tasks;
  if (t >= a.T) return;
  const int kind_task = (int)(task - t * tasks);
  const bool is_q = kind_task < q_tasks;
  const int first = is_q ? kind_task * per_q : (kind_task - q_tasks) * per_k;
  const int end = is_q ? min(first + per_q, a.Hq) : min(first + per_k, a.Hkv);
  const Lane at = lane_of<D>(a, lane);
  const void* wp = is_q ? a.w_q : a.w_k;
  const bool normed = wp != nullptr;
  const __nv_bfloat16* in = static_cast<const __nv_bfloat16*>(is_q ? a.q_in : a.k_in) +
                            t * (is_q ? a.q_row : a.k_row) + 8 * at.l;
  const int64_t step = is_q ? a.q_head : a.k_head;
  Weights w;
  Angles g;
  load_angles(g, a, position(a, t), at);
  load_weights(w, a, wp, at);
  float2 c[4], s[4];  // factors of the columns and of their partners, the weights among them
  auto factors = [&]() {
    float cc[8], ss[8];
    spread_angles(cc, ss, g, at, a.interleaved);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = make_float2(cc[2 * i] * w.own[2 * i], cc[2 * i + 1] * w.own[2 * i + 1]);
      s[i] = make_float2(ss[2 * i] * w.other[2 * i], ss[2 * i + 1] * w.other[2 * i + 1]);
    }
  };
  if (is_q || !a.cache) {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(is_q ? a.q_out : a.k_out) +
                         t * (is_q ? a.q_out_row : a.k_out_row) + 8 * at.l;
    const int64_t out_step = is_q ? a.q_out_head : a.k_out_head;
    uint4 raw[kUnroll];
    auto load = [&](int base) {
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = base + u * kHeads + side;
        raw[u] = h < end ? *reinterpret_cast<const uint4*>(in + h * step) : make_uint4(0, 0, 0, 0);
      }
    };
    load(first);
    factors();
#pragma unroll 1
    for (int base = first; base < end; base += kUnroll * kHeads) {
      uint4 now[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) now[u] = raw[u];
      load(base + kUnroll * kHeads);
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (base + u * kHeads >= end) break;  // (the same for the whole warp)
        float2 y[4];
        norm_rotate<D>(y, now[u], partners(now[u], at.from, at.turned, a.interleaved), normed, c, s, a.eps);
        const int h = base + u * kHeads + side;
        if (h < end)
          *reinterpret_cast<uint4*>(out + h * out_step) = make_uint4(pack2(y[0]), pack2(y[1]), pack2(y[2]), pack2(y[3]));
      }
    }
    return;
  }

  const __nv_bfloat16* vin = static_cast<const __nv_bfloat16*>(a.v_in) + t * a.v_row + 8 * at.l;
  const int64_t head_bytes = (int64_t)(a.page_size / kCacheBlock) * cache_block_bytes(D);
  uint4 next_raw, next_vals;
  auto load = [&](int h) {
    next_raw = h < end ? *reinterpret_cast<const uint4*>(in + h * step) : make_uint4(0, 0, 0, 0);
    next_vals = h < end ? *reinterpret_cast<const uint4*>(vin + h * a.v_head) : make_uint4(0, 0, 0, 0);
  };
  load(first + side);
  factors();
  const int64_t slot = a.slots[t];
  // What FP32 may be off by: with |x| <= sqrt(D) after the norm, half of 13
  // additions' and the root's three units, four products and a division,
  // below 2^-20 of sqrt(D) (|c w| + |s w'|); twice that, for the slack between.
  float off = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    off = fmaxf(off, fmaxf(fabsf(c[j].x) + fabsf(s[j].x), fabsf(c[j].y) + fabsf(s[j].y)));
  off = fmaxf(off, __shfl_xor_sync(0xffffffffu, off, 1));
  off *= 0x1p-19f * (D == 64 ? 8.f : D == 128 ? 11.4f : 16.f) / a.k_scale;
  const bool kept = slot >= 0 && slot < (int64_t)a.pages * a.page_size;
  const CachePlace place = cache_place(kept ? slot : 0, 0, a.Hkv, a.page_size, D);
  uint8_t* codes = static_cast<uint8_t*>(a.cache) + place.codes + 4 * at.l;
  uint8_t* scales = static_cast<uint8_t*>(a.cache) + place.scales + at.l / 2;
  unsigned again = 0;  // iterations whose keys' codes are open
#pragma unroll 1
  for (int base = first; base < end; base += kHeads) {
    const int h = base + side;
    const uint4 raw = next_raw, vals = next_vals;
    load(h + kHeads);
    const uint4 other = partners(raw, at.from, at.turned, a.interleaved);
    Quantised k, v;
    float2 u[4];
    norm_rotate<D>(u, raw, other, normed, c, s, a.eps);
    divide8(u, a.k_scale);
    const bool sure = quantise8<true>(u, off, k) && normed;
    again |= (__any_sync(0xffffffffu, !sure) ? 1u : 0u) << ((base - first) / kHeads);
    float x[8];
    unpack8(vals, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) u[j] = make_float2(x[2 * j], x[2 * j + 1]);
    divide8(u, a.v_scale);
    quantise8<false>(u, 0.f, v);
    if (head_any<D>(k.bad || v.bad, side)) k.scale = 0x7fu;
    if (h < end && kept) {
      const int64_t head = h * head_bytes;
      *reinterpret_cast<uint32_t*>(codes + head) = k.codes;
      *reinterpret_cast<uint32_t*>(codes + head + cache_half_bytes(D)) = v.codes;
      if (at.l % 2 == 0) {
        scales[head] = (uint8_t)k.scale;
        scales[head + cache_half_bytes(D)] = (uint8_t)v.scale;
      }
    }
  }
#pragma unroll 1
  for (; again; again &= again - 1) {
    const int h = first + (__ffs(again) - 1) * kHeads + side;
    const uint4 raw = h < end ? *reinterpret_cast<const uint4*>(in + h * step) : make_uint4(0, 0, 0, 0);
    const uint4 vals = h < end ? *reinterpret_cast<const uint4*>(vin + h * a.v_head) : make_uint4(0, 0, 0, 0);
    Quantised k;
    float2 u[4];
    norm_rotate_pairs<D>(u, a, t, raw, partners(raw, at.from, at.turned, a.interleaved), at);
    divide8(u, a.k_scale);
    quantise8<false>(u, 0.f, k);
    float x[8], top = 0.f;
    unpack8(vals, x);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(__fdiv_rn(x[i], a.v_scale)));
    if (head_any<D>(k.bad || !(top < INFINITY), side)) k.scale = 0x7fu;
    if (h < end && kept) {
      *reinterpret_cast<uint32_t*>(codes + h * head_bytes) = k.codes;
      if (at.l % 2 == 0) scales[h * head_bytes] = (uint8_t)k.scale;
    }
  }
}

template <int D>
cudaError_t launch_dim(const moe_fp4_qk_norm_rope_args& a, cudaStream_t st) {
  constexpr int kHeads = 32 / (D / 8), kAtOnce = kUnroll * kHeads;
  int sms = 0;
  const cudaError_t e = current_device_sms(&sms);
  if (e != cudaSuccess) return e;
  // few tokens: a task of what a warp has under way; many: all heads of a kind,
  // so that weights and angles are read once
  const bool many = a.T >= 16 * sms;
  const int per_q = many ? ceil_div(a.Hq, kAtOnce) * kAtOnce : kAtOnce;
  const int per_k = !a.cache ? per_q : many ? min(ceil_div(a.Hkv, kHeads), 32) * kHeads : kHeads;
  const int q_tasks = ceil_div(a.Hq, per_q), tasks = q_tasks + ceil_div(a.Hkv, per_k);
  const int64_t warps = (int64_t)a.T * tasks;
  const int64_t grid = (warps + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
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
