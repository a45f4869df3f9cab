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
#include <cstdlib>
#include "block.cuh"
#include "fp8_quant.cuh"
#include "host.cuh"

namespace moe_fp4 {

// Eight consecutive values from p + k (kVec: 16-byte aligned and k + 8 <= H),
// zeros past H.
template <bool kVec>
__device__ __forceinline__ void load8(const void* p, int f32, int64_t base, int k, int H, float (&v)[8]) {
  if (kVec) {
    if (f32) {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + base + k);
      const float4 a = q[0], b = q[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + base + k);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.f;
      if (k + i < H)
        v[i] = f32 ? static_cast<const float*>(p)[base + k + i]
                   : __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[base + k + i] << 16);
    }
  }
}

__device__ __forceinline__ uint32_t bf16x2_bits(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool kVec>
__device__ __forceinline__ void store8(void* p, int f32, int64_t base, int k, int H, const float (&v)[8]) {
  if (kVec) {
    if (f32) {
      float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + base + k);
      q[0] = make_float4(v[0], v[1], v[2], v[3]);
      q[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + base + k) = make_uint4(
          bf16x2_bits(v[0], v[1]), bf16x2_bits(v[2], v[3]), bf16x2_bits(v[4], v[5]), bf16x2_bits(v[6], v[7]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (k + i < H) {
        if (f32)
          static_cast<float*>(p)[base + k + i] = v[i];
        else
          static_cast<__nv_bfloat16*>(p)[base + k + i] = __float2bfloat16_rn(v[i]);
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

// Eight residual values as loaded: packed (bf16) or not (f32).
template <bool kF32>
struct Raw8 {
  uint32_t w[kF32 ? 8 : 4];
  template <bool kVec>
  __device__ __forceinline__ void load(const void* p, int64_t base, int k, int H) {
    if (kVec) {
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + (base + k) * (kF32 ? 4 : 2));
#pragma unroll
      for (int i = 0; i < (kF32 ? 2 : 1); ++i) {
        uint4 u;
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                     : "l"(q + i)
                     : "memory");
        w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
      }
    } else {
      float v[8];
      load8<false>(p, kF32, base, k, H, v);
#pragma unroll
      for (int i = 0; i < (kF32 ? 8 : 4); ++i)
        w[i] = kF32 ? __float_as_uint(v[i])
                    : (__float_as_uint(v[2 * i]) >> 16) | (__float_as_uint(v[2 * i + 1]) & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (kF32 ? 8 : 4); ++i) w[i] = 0;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = kF32 ? __uint_as_float(w[i])
                  : __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  }
};

// kCh chunks of eight columns per thread: chunk c = threadIdx.x + i *
// blockDim.x covers columns 8c .. 8c + 7.  All of a row's loads are under way
// before the first sum.
template <int kCh, int kMaxThreads, bool kVec, bool kF32>
__global__ void __launch_bounds__(kMaxThreads) block_norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float part[2][32];
  const int64_t m = blockIdx.x;
  const float inv_h = 1.0f / (float)a.H;
  Raw8<kF32> raw[kCh];
  Raw8<false> rawb[kCh];
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    const int k = 8 * (threadIdx.x + i * blockDim.x);
    raw[i].zero();
    rawb[i].zero();
    if (k < a.H) {
      if (a.b) rawb[i].template load<kVec>(a.b, m * a.b_row, k, a.H);
      raw[i].template load<kVec>(a.r, m * a.r_row, k, a.H);
    }
  }
  float v[kCh][8];  // r'
  if (a.b) {
    float inv = 1.f;
    if (a.w_post) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kCh; ++i) {
        float z[8];
        rawb[i].get(z);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += z[j] * z[j];
      }
      inv = rsqrtf(block_sum(sum, part[0]) * inv_h + a.eps);
    }
    float token_gate = 1.f;
    if (a.gate && a.g_col == 0)
      token_gate = a.g_f32 ? static_cast<const float*>(a.gate)[m * a.g_row]
                           : __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.gate)[m * a.g_row] << 16);
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      const int k = 8 * (threadIdx.x + i * blockDim.x);
      float z[8];
      rawb[i].get(z);
      raw[i].get(v[i]);
      if (k < a.H) {
        if (a.w_post) {
          float w[8];
          load8<kVec>(a.w_post, a.w_f32, 0, k, a.H, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) z[j] = z[j] * inv * (a.offset + w[j]);
        }
        if (a.gate && a.g_col) {
          float g[8];
          load8<kVec>(a.gate, a.g_f32, m * a.g_row, k, a.H, g);
#pragma unroll
          for (int j = 0; j < 8; ++j) z[j] *= g[j];
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) z[j] *= token_gate;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] += a.scale * z[j];
    }
  } else {
#pragma unroll
    for (int i = 0; i < kCh; ++i) raw[i].get(v[i]);
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    const int k = 8 * (threadIdx.x + i * blockDim.x);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += k + j < a.H ? v[i][j] * v[i][j] : 0.f;
    if (a.r_out && k < a.H) store8<kVec>(a.r_out, kF32, m * a.ro_row, k, a.H, v[i]);
  }
  if (!a.w_pre) return;
  const float inv = rsqrtf(block_sum(sum, part[1]) * inv_h + a.eps);
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    const int k = 8 * (threadIdx.x + i * blockDim.x);
    if (k < a.H) {
      float w[8];
      load8<kVec>(a.w_pre, a.w_f32, 0, k, a.H, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * inv * (a.offset + w[j]);
      if (a.n) store8<kVec>(a.n, 0, m * a.n_row, k, a.H, v[i]);
    }
    if (a.q) {
      // the BF16 values' FP8 form, so that it is the one a quantiser of n
      // gives; 16 lanes hold a block of 128 columns
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = k + j < a.H ? __bfloat162float(__float2bfloat16_rn(v[i][j])) : 0.f;
      const float sc = block_scale(block_amax(v[i]));
      if (k < a.H) {
        *reinterpret_cast<uint2*>(a.q + m * a.q_row + k) = e4m3_quotients(v[i], sc);
        if ((threadIdx.x & 15) == 0) a.s[m * a.s_row + (int64_t)(k / 128) * a.s_blk] = sc;
      }
    }
  }
}

template <int kCh, int kMaxThreads>
static cudaError_t launch_ch(const NormArgs& a, int res_f32, bool vec, cudaStream_t st) {
  const unsigned threads = (unsigned)((a.H + 256 * kCh - 1) / (256 * kCh)) * 32;
  const unsigned grid = (unsigned)a.M;
  if (vec && res_f32)
    block_norm_kernel<kCh, kMaxThreads, true, true><<<grid, threads, 0, st>>>(a);
  else if (vec)
    block_norm_kernel<kCh, kMaxThreads, true, false><<<grid, threads, 0, st>>>(a);
  else if (res_f32)
    block_norm_kernel<kCh, kMaxThreads, false, true><<<grid, threads, 0, st>>>(a);
  else
    block_norm_kernel<kCh, kMaxThreads, false, false><<<grid, threads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_block_norm(const NormArgs& a, int res_f32, bool vec, cudaStream_t st) {
  int sms = 0;
  const cudaError_t e = current_device_sms(&sms);
  if (e != cudaSuccess) return e;
  if (a.H > 16384) return launch_ch<4, 1024>(a, res_f32, vec, st);
  if (a.H > 8192) return launch_ch<4, 512>(a, res_f32, vec, st);
  if (getenv("NCH")) {
    int c = atoi(getenv("NCH"));
    if (c == 1) return launch_ch<1, 1024>(a, res_f32, vec, st);
    if (c == 2) return launch_ch<2, 512>(a, res_f32, vec, st);
    return launch_ch<4, 256>(a, res_f32, vec, st);
  }
  if (a.M <= sms) return launch_ch<1, 1024>(a, res_f32, vec, st);
  return launch_ch<4, 256>(a, res_f32, vec, st);
}

}  // namespace moe_fp4
