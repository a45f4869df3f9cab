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

// kCh chunks of eight columns per thread: chunk c = threadIdx.x + i *
// blockDim.x covers columns 8c .. 8c + 7.
template <int kCh, bool kVec>
__global__ void __launch_bounds__(1024) block_norm_kernel(NormArgs a, int res_f32) {
  __shared__ float part[2][32];
  const int64_t m = blockIdx.x;
  const float inv_h = 1.0f / (float)a.H;
  float v[kCh][8];  // r'
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    const int k = 8 * (threadIdx.x + i * blockDim.x);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
    if (k < a.H) load8<kVec>(a.r, res_f32, m * a.r_row, k, a.H, v[i]);
  }
  if (a.b) {
    float z[kCh][8];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      const int k = 8 * (threadIdx.x + i * blockDim.x);
#pragma unroll
      for (int j = 0; j < 8; ++j) z[i][j] = 0.f;
      if (k < a.H) load8<kVec>(a.b, 0, m * a.b_row, k, a.H, z[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += z[i][j] * z[i][j];
    }
    float inv = 1.f;
    if (a.w_post) inv = rsqrtf(block_sum(sum, part[0]) * inv_h + a.eps);
    const float token_gate =
        a.gate && a.g_col == 0
            ? (a.g_f32 ? static_cast<const float*>(a.gate)[m * a.g_row]
                       : __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.gate)[m * a.g_row] << 16))
            : 1.f;
#pragma unroll
    for (int i = 0; i < kCh; ++i) {
      const int k = 8 * (threadIdx.x + i * blockDim.x);
      if (k >= a.H) continue;
      if (a.w_post) {
        float w[8];
        load8<kVec>(a.w_post, a.w_f32, 0, k, a.H, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[i][j] = z[i][j] * inv * (a.offset + w[j]);
      }
      if (a.gate) {
        float g[8];
        if (a.g_col) load8<kVec>(a.gate, a.g_f32, m * a.g_row, k, a.H, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) z[i][j] *= a.g_col ? g[j] : token_gate;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] += a.scale * z[i][j];
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kCh; ++i) {
    const int k = 8 * (threadIdx.x + i * blockDim.x);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += k + j < a.H ? v[i][j] * v[i][j] : 0.f;
    if (a.r_out && k < a.H) store8<kVec>(a.r_out, res_f32, m * a.ro_row, k, a.H, v[i]);
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

template <int kCh>
static cudaError_t launch_ch(const NormArgs& a, int res_f32, bool vec, unsigned threads, cudaStream_t st) {
  if (vec)
    block_norm_kernel<kCh, true><<<(unsigned)a.M, threads, 0, st>>>(a, res_f32);
  else
    block_norm_kernel<kCh, false><<<(unsigned)a.M, threads, 0, st>>>(a, res_f32);
  return cudaGetLastError();
}

cudaError_t launch_block_norm(const NormArgs& a, int res_f32, bool vec, cudaStream_t st) {
  const int chunks = (a.H + 7) / 8;
  const int ch = chunks <= 1024 ? 1 : chunks <= 2048 ? 2 : 4;
  const unsigned threads = (unsigned)((chunks + 32 * ch - 1) / (32 * ch)) * 32;
  if (ch == 1) return launch_ch<1>(a, res_f32, vec, threads, st);
  if (ch == 2) return launch_ch<2>(a, res_f32, vec, threads, st);
  return launch_ch<4>(a, res_f32, vec, threads, st);
}

}  // namespace moe_fp4
