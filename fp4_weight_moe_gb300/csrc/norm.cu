// The norms before and after a block with its gate and residual scale
// (moe_fp4_block_norm):
//   z  = b * rsqrt(mean(b^2) + eps) * (o + w_post)   (z = b without w_post)
//   r' = r + scale * gate * z
//   n  = r' * rsqrt(mean(r'^2) + eps) * (o + w_pre)
// and n's FP8 form (a scale per 128 columns), in one launch.  A CTA (a warp)
// holds a row in registers, so b and r are read and r' and n written once; two
// sums over the row (of b^2, then of r'^2) are all that separates them.  Sums,
// r' and the norms are FP32; r' enters the second norm before it is rounded to
// the residual stream's type.
//
// Bound: HBM where rows are many and their starts alike (16384 x 7168, bf16
// residual, no norm after the block: 136 us, 6.9 TB/s of a copy's 6.8; f32
// residual, both norms, a gate per value: 244 us, 6.7; 4096 x 4096, both
// norms: 24 us, 5.6, with the FP8 form 29).  Odd widths pay for the weights,
// which do not shift with the rows and are read one by one (9000 x 5005, bf16,
// no norm after the block: 70 us, 5.1 TB/s, with it 90; with all rows read one
// by one 180).  Past 16384 columns one CTA of 1024 threads fills an SM's
// registers, so nothing runs beside a row's sums, and the odd forms and the FP32
// one spill some (1000 x 32768, both norms: 61 us, 4.3 TB/s, f32 97; 1000 x
// 32767 144).  Up to a few hundred rows the launch and the chain of two sums (64
// x 7168, f32, both norms: 3.7 us; one row of 2560 2.0).
#include "block.cuh"
#include "fp8_quant.cuh"
#include "host.cuh"

namespace moe_fp4 {

// How a row's columns lie on its threads (a chunk: eight columns of each):
//   kPacked   rows 16-byte aligned, H % 8 == 0: columns 8 (t + i T) .. + 7 of
//             chunk i, in 16-byte accesses;
//   kShifted  all rows' starts off a 16-byte boundary by the same `shift`
//             elements (contiguous rows of an odd width): the same, `shift`
//             columns earlier, so that accesses are aligned; the first and the
//             last eight are accessed one by one;
//   kSingle   the rest: columns t + (8 i + j) T, one by one, a warp's next to
//             each other.
// T threads to a row, t = 0 .. T - 1.  Columns outside the row read as zeros
// and are not stored.
enum Layout { kPacked, kShifted, kSingle };

struct Place {
  int t, T, shift, H;
  template <Layout kL>
  __device__ __forceinline__ int column(int i, int j) const {
    return kL == kSingle ? t + (8 * i + j) * T : 8 * (t + i * T) + j - (kL == kShifted ? shift : 0);
  }
  __device__ __forceinline__ bool holds(int c) const { return (unsigned)c < (unsigned)H; }
  // all eight of the chunk in the row
  template <Layout kL>
  __device__ __forceinline__ bool whole(int i) const {
    if (kL == kSingle) return false;
    const int c = column<kL>(i, 0);
    return kL == kPacked ? c < H : c >= 0 && c + 8 <= H;
  }
};

__device__ __forceinline__ uint4 ld_once(const void* p) {  // read once, not worth a line of L1
  uint4 u;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p)
               : "memory");
  return u;
}

// Eight bf16 (kF32: f32) values of a row as loaded, packed.
template <bool kF32>
struct Raw8 {
  uint32_t w[kF32 ? 8 : 4];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (kF32 ? 8 : 4); ++i) w[i] = 0;
  }
  __device__ __forceinline__ void put(int c, uint4 u) { w[4 * c] = u.x, w[4 * c + 1] = u.y, w[4 * c + 2] = u.z, w[4 * c + 3] = u.w; }
  // kVector: one of the weights, which start at a 16-byte boundary (if
  // kPacked) whatever the rows' shift.
  template <Layout kL, bool kVector>
  __device__ __forceinline__ void load(const void* row, int i, const Place& p) {
    if (p.whole<kL>(i) && (kL == kPacked || !kVector)) {
      const char* q = static_cast<const char*>(row) + (int64_t)p.column<kL>(i, 0) * (kF32 ? 4 : 2);
#pragma unroll
      for (int c = 0; c < (kF32 ? 2 : 1); ++c)
        put(c, kVector ? reinterpret_cast<const uint4*>(q)[c] : ld_once(q + 16 * c));
    } else if (kL != kPacked) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = p.column<kL>(i, j);
        uint32_t u = 0;
        if (p.holds(k))
          u = kF32 ? static_cast<const uint32_t*>(row)[k] : (uint32_t) static_cast<const uint16_t*>(row)[k];
        if (kF32)
          w[j] = u;
        else if (j % 2 == 0)
          w[j / 2] = u;
        else
          w[j / 2] |= u << 16;
      }
    }
  }
  __device__ __forceinline__ float2 pair(int p) const {
    return kF32 ? make_float2(__uint_as_float(w[2 * p]), __uint_as_float(w[2 * p + 1]))
                : make_float2(__uint_as_float(w[p] << 16), __uint_as_float(w[p] & 0xffff0000u));
  }
};

// The chunk's values of a weight or a row of either type.
template <Layout kL, bool kVector>
__device__ __forceinline__ void load_pairs(const void* row, int f32, int i, const Place& at, float2 (&v)[4]) {
  if (f32) {
    Raw8<true> r;
    r.zero();
    r.template load<kL, kVector>(row, i, at);
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = r.pair(p);
  } else {
    Raw8<false> r;
    r.zero();
    r.template load<kL, kVector>(row, i, at);
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = r.pair(p);
  }
}

__device__ __forceinline__ uint32_t bf16x2_bits(float2 v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <Layout kL, bool kF32>
__device__ __forceinline__ void store_pairs(void* row, int i, const Place& at, const float2 (&v)[4]) {
  if (at.whole<kL>(i)) {
    const int k = at.column<kL>(i, 0);
    if (kF32) {
      float4* q = reinterpret_cast<float4*>(static_cast<float*>(row) + k);
      q[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
      q[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + k) =
          make_uint4(bf16x2_bits(v[0]), bf16x2_bits(v[1]), bf16x2_bits(v[2]), bf16x2_bits(v[3]));
    }
  } else if (kL != kPacked) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = at.column<kL>(i, j);
      const float x = j % 2 ? v[j / 2].y : v[j / 2].x;
      if (at.holds(k)) {
        if (kF32)
          static_cast<float*>(row)[k] = x;
        else
          static_cast<__nv_bfloat16*>(row)[k] = __float2bfloat16_rn(x);
      }
    }
  }
}

// Sum over a row's threads: the warp, or the CTA (`part` has a slot per warp).
template <bool kWarp>
__device__ __forceinline__ float row_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warps = blockDim.x >> 5;
  if (kWarp || warps == 1) return v;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (int)(threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Weights or a gate on their way to a thread's own slots, slot[c T]: one a
// chunk, two of 32-bit values.
enum { kStageGate = 1, kStagePost = 2, kStagePre = 4 };

template <int kCh>
__device__ __host__ constexpr int staged_slots(int f32) { return f32 ? 2 * kCh : kCh; }

template <int kCh>
__device__ __forceinline__ void stage_row(uint4* slot, const void* row, int f32, const Place& at) {
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    const char* q = static_cast<const char*>(row) + (int64_t)at.column<kPacked>(i, 0) * (f32 ? 4 : 2);
    if (at.whole<kPacked>(i)) {
      cp_async_16(slot + (f32 ? 2 * i : i) * blockDim.x, q);
      if (f32) cp_async_16(slot + (2 * i + 1) * blockDim.x, q + 16);
    }
  }
}

__device__ __forceinline__ void staged_pairs(const uint4* slot, int f32, int i, const Place& at, float2 (&v)[4]) {
  Raw8<true> u;  // (zeros outside the row: what lies in memory there may be NaN)
  u.zero();
  if (at.whole<kPacked>(i)) {
    u.put(0, slot[(f32 ? 2 * i : i) * blockDim.x]);
    if (f32) u.put(1, slot[(2 * i + 1) * blockDim.x]);
  }
  Raw8<false> h;
  h.put(0, make_uint4(u.w[0], u.w[1], u.w[2], u.w[3]));
#pragma unroll
  for (int p = 0; p < 4; ++p) v[p] = f32 ? u.pair(p) : h.pair(p);
}

// Value `m` of a gate or the like, of either type.
__device__ __forceinline__ float scalar_of(const void* p, int f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i]
             : __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}

// A CTA or (kWarp) a warp per row, kCh chunks of eight columns per thread; all
// of a row's loads are under way before the first sum, those of weights and of
// a gate per value (packed rows, a.staged) on their way into shared memory, a
// thread's own values by itself.
// (CTAs per SM: as many as the loads in flight need, a bound on the registers)
constexpr int resident(int chunks, int threads, Layout layout, bool f32, bool warp) {
  if (threads != 256 || layout == kSingle) return 1;
  if (chunks == 4) return f32 ? 3 : 4;
  return chunks == 2 ? (warp || f32 ? 4 : 5) : 6;
}

template <int kCh, int kMaxThreads, Layout kL, bool kF32, bool kWarp>
__global__ void __launch_bounds__(kMaxThreads, resident(kCh, kMaxThreads, kL, kF32, kWarp)) block_norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float part[2][32];
  pdl_wait();
  pdl_launch_dependents();
  extern __shared__ uint4 stage[];
  const int64_t m = kWarp ? (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
  if (kWarp && m >= a.M) return;
  const int H = a.H;
  const Place at = {kWarp ? (int)threadIdx.x & 31 : (int)threadIdx.x, kWarp ? 32 : (int)blockDim.x,
                    kL == kShifted ? (a.shift + (int)(m & 7) * a.shift_row) & 7 : 0, H};
  const float inv_h = 1.0f / (float)H;
  Raw8<kF32> raw[kCh];
  Raw8<false> rawb[kCh];
  const uint16_t* b = a.b ? a.b + m * a.b_row : nullptr;
  const void* r = static_cast<const char*>(a.r) + m * a.r_row * (kF32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    raw[i].zero();
    rawb[i].zero();
    if (b) rawb[i].template load<kL, false>(b, i, at);
    raw[i].template load<kL, false>(r, i, at);
  }
  const char* gate = static_cast<const char*>(a.gate);
  float factor = a.scale;  // what the row's values of z share
  if (gate && a.g_col)
    gate += m * a.g_row * (a.g_f32 ? 4 : 2);
  else if (gate)
    factor *= scalar_of(gate, a.g_f32, m * a.g_row);
  const int staged = kL == kPacked ? a.staged : 0;
  uint4* const s_gate = stage + threadIdx.x;
  uint4* const s_post = s_gate + (staged & kStageGate ? staged_slots<kCh>(a.g_f32) * blockDim.x : 0);
  uint4* const s_pre = s_post + (staged & kStagePost ? staged_slots<kCh>(a.w_f32) * blockDim.x : 0);
  if (staged) {
    if (staged & kStageGate) stage_row<kCh>(s_gate, gate, a.g_f32, at);
    if (staged & kStagePost) stage_row<kCh>(s_post, a.w_post, a.w_f32, at);
    cp_async_commit();
    if (staged & kStagePre) stage_row<kCh>(s_pre, a.w_pre, a.w_f32, at);
    cp_async_commit();
  }
  float2 v[kCh][4];  // r'
  if (b) {
    if (a.w_post) {
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kCh; ++i)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float2 z = rawb[i].pair(p);
          sum = ffma2(z, z, sum);
        }
      factor *= rsqrtf(row_sum<kWarp>(sum.x + sum.y, part[0]) * inv_h + a.eps);
    }
    const float2 f = make_float2(factor, factor);
    const float2 of = make_float2(a.offset * factor, a.offset * factor);
    if (staged) cp_async_wait<1>();
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      float2 t[4];  // factor * (offset + w_post) * gate
#pragma unroll
      for (int p = 0; p < 4; ++p) t[p] = f;
      if (a.w_post) {
        float2 w[4];
        if (staged & kStagePost)
          staged_pairs(s_post, a.w_f32, i, at, w);
        else
          load_pairs<kL, true>(a.w_post, a.w_f32, i, at, w);
#pragma unroll
        for (int p = 0; p < 4; ++p) t[p] = ffma2(w[p], f, of);
      }
      if (a.gate && a.g_col) {
        float2 g[4];
        if (staged & kStageGate) {
          staged_pairs(s_gate, a.g_f32, i, at, g);
        } else if (a.g_row == 0 && kL == kShifted) {  // one gate for all rows, which does not shift with them
          load_pairs<kL, true>(gate, a.g_f32, i, at, g);
        } else {
          load_pairs<kL, false>(gate, a.g_f32, i, at, g);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) t[p] = fmul2(t[p], g[p]);
      }
#pragma unroll
      for (int p = 0; p < 4; ++p) v[i][p] = ffma2(rawb[i].pair(p), t[p], raw[i].pair(p));
    }
  } else {
#pragma unroll
    for (int i = 0; i < kCh; ++i)
#pragma unroll
      for (int p = 0; p < 4; ++p) v[i][p] = raw[i].pair(p);
  }
  if (a.r_out) {
    void* row = static_cast<char*>(a.r_out) + m * a.ro_row * (kF32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < kCh; ++i) store_pairs<kL, kF32>(row, i, at, v[i]);
  }
  if (!a.w_pre) return;
  float2 sum = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kCh; ++i)
#pragma unroll
    for (int p = 0; p < 4; ++p) sum = ffma2(v[i][p], v[i][p], sum);  // (columns past H are zeros)
  const float inv = rsqrtf(row_sum<kWarp>(sum.x + sum.y, part[1]) * inv_h + a.eps);
  const float2 f = make_float2(inv, inv), of = make_float2(a.offset * inv, a.offset * inv);
  if (staged) cp_async_wait<0>();
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    float2 w[4];
    if (staged & kStagePre)
      staged_pairs(s_pre, a.w_f32, i, at, w);
    else
      load_pairs<kL, true>(a.w_pre, a.w_f32, i, at, w);
#pragma unroll
    for (int p = 0; p < 4; ++p) v[i][p] = fmul2(v[i][p], ffma2(w[p], f, of));
    if (a.n) store_pairs<kL, false>(a.n + m * a.n_row, i, at, v[i]);
    if (kL == kPacked && a.q) {
      // the BF16 values' FP8 form, so that it is the one a quantiser of n
      // gives; 16 lanes hold a block of 128 columns
      const int k = at.column<kL>(i, 0);
      float x[8];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint32_t u = bf16x2_bits(v[i][p]);
        x[2 * p] = __uint_as_float(u << 16);
        x[2 * p + 1] = __uint_as_float(u & 0xffff0000u);
      }
      const float sc = block_scale(block_amax(x));
      if (k < H) {
        *reinterpret_cast<uint2*>(a.q + m * a.q_row + k) = e4m3_quotients(x, sc);
        if ((at.t & 15) == 0) a.s[m * a.s_row + (int64_t)(k / 128) * a.s_blk] = sc;
      }
    }
  }
}

template <int kCh, int kMaxThreads, bool kWarp>
static cudaError_t launch_ch(NormArgs a, int res_f32, cudaStream_t st) {
  const int columns = a.H + (a.layout == kShifted ? 7 : 0);
  const unsigned threads = kWarp ? kMaxThreads : (unsigned)((columns + 256 * kCh - 1) / (256 * kCh)) * 32;
  const unsigned grid = kWarp ? (unsigned)(((int64_t)a.M + kMaxThreads / 32 - 1) / (kMaxThreads / 32)) : (unsigned)a.M;
  // Staged while 48 KB hold it (what a launch gets unasked), the gate first,
  // whose values come from memory; not the weights of a warp's row, which the
  // CTA's other rows leave in L1 (16384 x 264 8.2 us, staged 10.2; a row per
  // CTA: 9000 x 5120, f32, a gate per value 125 us, staged 98).
  size_t smem = 0;
  a.staged = 0;
  auto stage = [&](int what, int f32) {
    const size_t more = (size_t)staged_slots<kCh>(f32) * threads * 16;
    if (smem + more <= 47 * 1024) smem += more, a.staged |= what;
  };
  if (a.layout == kPacked) {
    if (a.gate && a.g_col) stage(kStageGate, a.g_f32);
    if (!kWarp && a.w_post) stage(kStagePost, a.w_f32);
    if (!kWarp && a.w_pre) stage(kStagePre, a.w_f32);
  }
  auto* kern = a.layout == kPacked ? (res_f32 ? block_norm_kernel<kCh, kMaxThreads, kPacked, true, kWarp>
                                              : block_norm_kernel<kCh, kMaxThreads, kPacked, false, kWarp>)
               : a.layout == kShifted ? (res_f32 ? block_norm_kernel<kCh, kMaxThreads, kShifted, true, kWarp>
                                                 : block_norm_kernel<kCh, kMaxThreads, kShifted, false, kWarp>)
                                      : (res_f32 ? block_norm_kernel<kCh, kMaxThreads, kSingle, true, kWarp>
                                                 : block_norm_kernel<kCh, kMaxThreads, kSingle, false, kWarp>);
  return launch_dependent_smem(kern, grid, threads, smem, st, a);
}

// kShifted where every array that is read or written by rows is off a 16-byte
// boundary by the same elements in every row (of 32-bit types: modulo four).
// An array with a single row for all tokens would not shift with the others.
static bool same_shift(const NormArgs& a, int res_f32, int* shift, int* shift_row) {
  int modulo = 0;  // of the values seen so far: 4, later 8
  *shift = *shift_row = 0;
  bool same = true;
  auto see = [&](const void* p, int64_t row, int f32) {
    if (!p) return;
    const int mod = f32 ? 4 : 8, bytes = f32 ? 4 : 2;
    const int s = (int)((uintptr_t)p / bytes % mod), r = (int)(row % mod);
    const int low = modulo && modulo < mod ? modulo : mod;
    same = same && (!modulo || (s % low == *shift % low && r % low == *shift_row % low));
    if (mod > modulo) modulo = mod, *shift = s, *shift_row = r;
  };
  see(a.r, a.r_row, res_f32);
  see(a.r_out, a.ro_row, res_f32);
  see(a.b, a.b_row, 0);
  see(a.n, a.n_row, 0);
  if (a.gate && a.g_col && a.g_row) see(a.gate, a.g_row, a.g_f32);
  return same && a.H + 7 <= 32768;  // (the threads hold 32768 columns)
}

cudaError_t launch_block_norm(NormArgs a, int res_f32, bool packed, cudaStream_t st) {
  int sms = 0;
  const cudaError_t e = current_device_sms(&sms);
  if (e != cudaSuccess) return e;
  a.layout = packed ? kPacked : same_shift(a, res_f32, &a.shift, &a.shift_row) ? kShifted : kSingle;
  const bool many = a.M > 2 * sms;
  const int columns = a.H + (a.layout == kShifted ? 7 : 0);
  if (columns > 16384) return launch_ch<4, 1024, false>(a, res_f32, st);
  if (columns > 8192) return launch_ch<4, 512, false>(a, res_f32, st);
  // A warp per row while two chunks of eight a lane hold it: no barrier, and
  // short rows leave no threads idle (16384 x 264 17.5 us with a CTA per row,
  // 8.3; with four chunks 16384 x 1024, f32, a gate per value: 37.9, 55.8).
  if (many && columns <= 256) return launch_ch<1, 256, true>(a, res_f32, st);
  if (many && columns <= 512) return launch_ch<2, 256, true>(a, res_f32, st);
  // Chunks per thread: one while a row per CTA leaves SMs with one or two
  // rows (latency) and where a row is short or read by scalar loads; beyond,
  // as many as keep a CTA at 256 threads, so that more rows share an SM and
  // their waits for the two sums overlap.  Measured with 1 / 2 / 4 chunks (us;
  // bf16 residual, no norm after the block): H=7168 M=64 2.5 / 2.5 / 3.0,
  // M=600 7.8 / 5.6 / 4.9, M=16384 231 / 154 / 136; H=4096 M=64 2.1 / 2.3 /
  // 2.8, M=16384 90 / 80 / 80; H=2560 M=16384 59 / 51 / 52; f32 residual with
  // that norm, M=16384: H=7168 383 / 251 / 224, H=4096 169 / 129 / 122, H=2560
  // 88 / 79 / 81.
  if (a.layout == kSingle || columns <= 2048 || !many) return launch_ch<1, 1024, false>(a, res_f32, st);
  if (columns <= 4096) return launch_ch<2, 256, false>(a, res_f32, st);
  return launch_ch<4, 256, false>(a, res_f32, st);
}

}  // namespace moe_fp4
