// The norms before and after a block with its gate and residual scale
// (moe_fp4_block_norm):
//   z  = b * rsqrt(mean(b^2) + eps) * (o + w_post)   (z = b without w_post)
//   r' = r + scale * gate * z
//   n  = r' * rsqrt(mean(r'^2) + eps) * (o + w_pre)
// and n's FP8 form (a scale per 128 columns), in one launch.  HBM bound: a
// CTA holds a row in registers, so b and r are read and r' and n written
// once; two block sums (of b^2, then of r'^2) are all that separates them.
// Sums, r' and the norms are FP32; r' enters the second norm before it is
// rounded to the residual stream's type.
#include "block.cuh"
#include "fp8_quant.cuh"
#include "host.cuh"

namespace moe_fp4 {

// A thread's eight columns of chunk i.  kVec (rows 16-byte aligned, H % 8 ==
// 0): eight consecutive ones from 8 (threadIdx.x + i blockDim.x).  Otherwise
// columns threadIdx.x + (8 i + j) blockDim.x, so that a warp's scalar
// accesses are consecutive.  Columns past H read as zeros and are not stored.
template <bool kVec>
__device__ __forceinline__ int column(int i, int j) {
  return kVec ? 8 * (threadIdx.x + i * blockDim.x) + j : (int)(threadIdx.x + (8 * i + j) * blockDim.x);
}

// Eight bf16 (kF32: f32) values of a row as loaded, packed.
template <bool kF32>
struct Raw8 {
  uint32_t w[kF32 ? 8 : 4];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (kF32 ? 8 : 4); ++i) w[i] = 0;
  }
  // kStream: read once, not worth a line of L1.
  template <bool kVec, bool kStream>
  __device__ __forceinline__ void load(const void* row, int i, int H) {
    if (kVec) {
      const int k = column<true>(i, 0);
      if (k >= H) return;
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(row) + (int64_t)k * (kF32 ? 4 : 2));
#pragma unroll
      for (int c = 0; c < (kF32 ? 2 : 1); ++c) {
        uint4 u;
        if (kStream)
          asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                       : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                       : "l"(q + c)
                       : "memory");
        else
          u = q[c];
        w[4 * c] = u.x, w[4 * c + 1] = u.y, w[4 * c + 2] = u.z, w[4 * c + 3] = u.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int k = column<false>(i, j);
        uint32_t u = 0;
        if (k < H) u = kF32 ? static_cast<const uint32_t*>(row)[k] : (uint32_t) static_cast<const uint16_t*>(row)[k];
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

// The chunk's values of a vector or row of either type.
template <bool kVec>
__device__ __forceinline__ void load_pairs(const void* row, int f32, int i, int H, float2 (&v)[4]) {
  if (f32) {
    Raw8<true> r;
    r.zero();
    r.template load<kVec, false>(row, i, H);
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = r.pair(p);
  } else {
    Raw8<false> r;
    r.zero();
    r.template load<kVec, false>(row, i, H);
#pragma unroll
    for (int p = 0; p < 4; ++p) v[p] = r.pair(p);
  }
}

__device__ __forceinline__ uint32_t bf16x2_bits(float2 v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool kVec, bool kF32>
__device__ __forceinline__ void store_pairs(void* row, int i, int H, const float2 (&v)[4]) {
  if (kVec) {
    const int k = column<true>(i, 0);
    if (k >= H) return;
    if (kF32) {
      float4* q = reinterpret_cast<float4*>(static_cast<float*>(row) + k);
      q[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
      q[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + k) =
          make_uint4(bf16x2_bits(v[0]), bf16x2_bits(v[1]), bf16x2_bits(v[2]), bf16x2_bits(v[3]));
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int k = column<false>(i, j);
      const float x = j % 2 ? v[j / 2].y : v[j / 2].x;
      if (k < H) {
        if (kF32)
          static_cast<float*>(row)[k] = x;
        else
          static_cast<__nv_bfloat16*>(row)[k] = __float2bfloat16_rn(x);
      }
    }
  }
}

// Sum over the CTA; `part` has a slot per warp.
__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (int)(threadIdx.x & 31) < warps ? part[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Value `m` of a gate or the like, of either type.
__device__ __forceinline__ float scalar_of(const void* p, int f32, int64_t i) {
  return f32 ? static_cast<const float*>(p)[i]
             : __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
}

// A CTA per row, kCh chunks of eight columns per thread; all of a row's loads
// are under way before the first sum.
template <int kCh, int kMaxThreads, bool kVec, bool kF32>
__global__ void __launch_bounds__(kMaxThreads) block_norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float part[2][32];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t m = blockIdx.x;
  const int H = a.H;
  const float inv_h = 1.0f / (float)H;
  Raw8<kF32> raw[kCh];
  Raw8<false> rawb[kCh];
  const uint16_t* b = a.b ? a.b + m * a.b_row : nullptr;
  const void* r = static_cast<const char*>(a.r) + m * a.r_row * (kF32 ? 4 : 2);
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    raw[i].zero();
    rawb[i].zero();
    if (b) rawb[i].template load<kVec, true>(b, i, H);
    raw[i].template load<kVec, true>(r, i, H);
  }
  float2 v[kCh][4];  // r'
  if (b) {
    float factor = a.scale;  // what the row's values of z share
    if (a.w_post) {
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kCh; ++i)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float2 z = rawb[i].pair(p);
          sum = ffma2(z, z, sum);
        }
      factor *= rsqrtf(block_sum(sum.x + sum.y, part[0]) * inv_h + a.eps);
    }
    if (a.gate && a.g_col == 0) factor *= scalar_of(a.gate, a.g_f32, m * a.g_row);
    const float2 f = make_float2(factor, factor);
    const float2 of = make_float2(a.offset * factor, a.offset * factor);
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      float2 t[4];  // factor * (offset + w_post) * gate
#pragma unroll
      for (int p = 0; p < 4; ++p) t[p] = f;
      if (a.w_post) {
        float2 w[4];
        load_pairs<kVec>(a.w_post, a.w_f32, i, H, w);
#pragma unroll
        for (int p = 0; p < 4; ++p) t[p] = ffma2(w[p], f, of);
      }
      if (a.gate && a.g_col) {
        float2 g[4];
        load_pairs<kVec>(static_cast<const char*>(a.gate) + m * a.g_row * (a.g_f32 ? 4 : 2), a.g_f32, i, H, g);
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
    for (int i = 0; i < kCh; ++i) store_pairs<kVec, kF32>(row, i, H, v[i]);
  }
  if (!a.w_pre) return;
  float2 sum = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < kCh; ++i)
#pragma unroll
    for (int p = 0; p < 4; ++p) sum = ffma2(v[i][p], v[i][p], sum);  // (columns past H are zeros)
  const float inv = rsqrtf(block_sum(sum.x + sum.y, part[1]) * inv_h + a.eps);
  const float2 f = make_float2(inv, inv), of = make_float2(a.offset * inv, a.offset * inv);
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    float2 w[4];
    load_pairs<kVec>(a.w_pre, a.w_f32, i, H, w);
#pragma unroll
    for (int p = 0; p < 4; ++p) v[i][p] = fmul2(v[i][p], ffma2(w[p], f, of));
    if (a.n) store_pairs<kVec, false>(a.n + m * a.n_row, i, H, v[i]);
    if (kVec && a.q) {
      // the BF16 values' FP8 form, so that it is the one a quantiser of n
      // gives; 16 lanes hold a block of 128 columns
      const int k = column<true>(i, 0);
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
        if ((threadIdx.x & 15) == 0) a.s[m * a.s_row + (int64_t)(k / 128) * a.s_blk] = sc;
      }
    }
  }
}

template <int kCh, int kMaxThreads>
static cudaError_t launch_ch(const NormArgs& a, int res_f32, bool vec, cudaStream_t st) {
  const unsigned threads = (unsigned)((a.H + 256 * kCh - 1) / (256 * kCh)) * 32;
  auto* kern = vec ? (res_f32 ? block_norm_kernel<kCh, kMaxThreads, true, true>
                              : block_norm_kernel<kCh, kMaxThreads, true, false>)
                   : (res_f32 ? block_norm_kernel<kCh, kMaxThreads, false, true>
                              : block_norm_kernel<kCh, kMaxThreads, false, false>);
  return launch_dependent(kern, (unsigned)a.M, threads, st, a);
}

cudaError_t launch_block_norm(const NormArgs& a, int res_f32, bool vec, cudaStream_t st) {
  int sms = 0;
  const cudaError_t e = current_device_sms(&sms);
  if (e != cudaSuccess) return e;
  if (a.H > 16384) return launch_ch<4, 1024>(a, res_f32, vec, st);
  if (a.H > 8192) return launch_ch<4, 512>(a, res_f32, vec, st);
  // Chunks per thread: one while a row per CTA leaves SMs with one or two
  // rows (latency) and where a row is short or read by scalar loads; beyond,
  // as many as keep a CTA at 256 threads, so that more rows share an SM and
  // their waits for the two sums overlap.  Measured with 1 / 2 / 4 chunks
  // (us, bf16 residual, no norm after the block): H=7168 M=64 2.5 / - / 3.3,
  // M=16384 151 / - / 138; H=4096 M=64 2.3 / 2.6 / 3.3, M=16384 81.4 / 80.0 /
  // 80.7; f32 residual with that norm, M=16384: H=7168 365 / - / 221, H=4096
  // 133 / 126 / 129, H=2560 85 / 77 / 81.
  if (!vec || a.H <= 2048 || a.M <= 2 * sms) return launch_ch<1, 1024>(a, res_f32, vec, st);
  if (a.H <= 4096) return launch_ch<2, 256>(a, res_f32, vec, st);
  return launch_ch<4, 256>(a, res_f32, vec, st);
}

}  // namespace moe_fp4
