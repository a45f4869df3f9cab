// FP8 products with a scale per block of 128 (moe_fp4_fp8_*): the activation
// quantiser and the launches of the product kernels of gemm_fp8.cuh.
#include "block.cuh"
#include "gemm_fp8.cuh"
#include "host.cuh"

namespace moe_fp4 {

// Status word of the product kernels' bounded waits (moe_fp4_fp8_status).
static __device__ uint32_t g_fp8_status;

cudaError_t fp8_status_address(void** p) { return cudaGetSymbolAddress(p, g_fp8_status); }

// ---------------------------------------------------------------- quantiser
// Per row and 128 columns: s = max|v| / 448 (1 where that is zero),
// q = e4m3_rn(v / s), each step an IEEE FP32 operation; v is the input, or
// act(gate) * up of a gated row [gate | up].  HBM bound: 16 lanes hold one
// block's 128 elements (16 bytes of BF16 each), so the block maximum is four
// shuffles and a block is read and written once.
__device__ __forceinline__ void bf16x8_to_float(uint4 u, float (&v)[8]) {
  const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(p[i] << 16);
    v[2 * i + 1] = __uint_as_float(p[i] & 0xffff0000u);
  }
}

// Four floats -> four E4M3 bytes (round to nearest even, saturating).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// SiLU in full FP32 precision: the scale of a block follows its largest
// product, and an element near the middle of two E4M3 values turns on it.
__device__ __forceinline__ float gated_exact(float g, float u, const ActParams& act) {
  if (act.kind == MOE_FP4_ACT_SILU) return g / (1.0f + expf(-g)) * u;
  return gated_act(g, u, act);
}

template <bool kGated>
__global__ void __launch_bounds__(256) fp8_quantize_kernel(const uint16_t* __restrict__ x, int64_t x_row, ActParams act,
                                                           uint8_t* __restrict__ q, int64_t q_row,
                                                           float* __restrict__ s, int64_t s_row, int64_t s_blk, int M,
                                                           int K) {
  const int nb = (K + 127) / 128;
  const int64_t units = (int64_t)M * nb;
  const int lane16 = threadIdx.x & 15;
  // the stride is a multiple of the two units of a warp, so a warp's 32 lanes
  // leave the loop together but for the last unit
  for (int64_t u = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / 16; u < ((units + 1) & ~(int64_t)1);
       u += (int64_t)gridDim.x * blockDim.x / 16) {
    const bool have = u < units;
    const int64_t m = have ? u / nb : 0;
    const int b = have ? (int)(u % nb) : 0;
    const int k = b * 128 + lane16 * 8;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (have && k < K) {
      bf16x8_to_float(*reinterpret_cast<const uint4*>(x + m * x_row + k), v);
      if (kGated) {
        float up[8];
        bf16x8_to_float(*reinterpret_cast<const uint4*>(x + m * x_row + K + k), up);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = gated_exact(v[i], up[i], act);
      }
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float sc = __fdiv_rn(amax, 448.f);
    if (sc == 0.f) sc = 1.f;  // an all-zero block, or one below FP32's reach
    if (have && k < K) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __fdiv_rn(v[i], sc);
      *reinterpret_cast<uint2*>(q + m * q_row + k) =
          make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
    }
    if (have && lane16 == 0) s[m * s_row + (int64_t)b * s_blk] = sc;
  }
}

cudaError_t launch_fp8_quantize(const void* x, int64_t x_row, const ActParams* act, void* q, int64_t q_row, float* s,
                                int64_t s_row, int64_t s_blk, int M, int K, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = current_device_sms(&sms);
  if (e != cudaSuccess) return e;
  const int64_t units = (int64_t)M * ((K + 127) / 128);
  const int64_t want = (units + 15) / 16, most = (int64_t)sms * 8;
  const unsigned grid = (unsigned)(want < most ? want : most);
  const ActParams none = {MOE_FP4_ACT_SILU, 0.f, 0.f, 0.f};
  if (act)
    fp8_quantize_kernel<true><<<grid, 256, 0, st>>>(static_cast<const uint16_t*>(x), x_row, *act,
                                                    static_cast<uint8_t*>(q), q_row, s, s_row, s_blk, M, K);
  else
    fp8_quantize_kernel<false><<<grid, 256, 0, st>>>(static_cast<const uint16_t*>(x), x_row, none,
                                                     static_cast<uint8_t*>(q), q_row, s, s_row, s_blk, M, K);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ product
template <int BN, bool kSwap>
__global__ void __launch_bounds__(F8Cfg<BN, kSwap>::kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, Fp8Args a) {
  a.err = &g_fp8_status;
  gemm_fp8_persistent<BN, kSwap>(&map_a, &map_b, a);
}

template <int BN, bool kSwap, bool kTwo>
__global__ void __launch_bounds__(F8Cfg<BN, kSwap, kTwo>::kThreads, kTwo ? 2 : 1)
    fp8_split_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, Fp8Args a,
                     int split) {
  a.err = &g_fp8_status;
  gemm_fp8_persistent<BN, kSwap, kTwo, true>(&map_a, &map_b, a, split);
}

struct Operands {
  const void *x, *w;
  int64_t x_row, w_row;
};

static cudaError_t encode(CUtensorMap* mx, CUtensorMap* mw, const Operands& o, const Fp8Args& a, int x_rows,
                          int w_rows) {
  CUresult r = encode_u8_map_2d(mx, o.x, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)o.x_row, (uint32_t)x_rows);
  if (r == CUDA_SUCCESS)
    r = encode_u8_map_2d(mw, o.w, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)o.w_row, (uint32_t)w_rows);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int BN, bool kSwap>
static cudaError_t launch_gemm(const Operands& o, const Fp8Args& a, int sms, cudaStream_t st) {
  using Cfg = F8Cfg<BN, kSwap>;
  CUtensorMap mx, mw;
  cudaError_t e = encode(&mx, &mw, o, a, Cfg::kXRows, Cfg::kWRows);
  static bool seen[64];
  if (e == cudaSuccess) e = allow_smem(fp8_gemm_kernel<BN, kSwap>, Cfg::kSmem, seen);
  if (e != cudaSuccess) return e;
  const int64_t tiles =
      (int64_t)((a.M + Cfg::kXRows - 1) / Cfg::kXRows) * ((a.N + Cfg::kWRows - 1) / Cfg::kWRows);
  const unsigned grid = (unsigned)(tiles < sms ? tiles : sms);
  fp8_gemm_kernel<BN, kSwap><<<grid, Cfg::kThreads, Cfg::kSmem, st>>>(kSwap ? mw : mx, kSwap ? mx : mw, a);
  return cudaGetLastError();
}

template <int BN, bool kSwap, bool kTwo>
static cudaError_t launch_split(const Operands& o, const Fp8Args& a, int tiles, int split, cudaStream_t st) {
  using Cfg = F8Cfg<BN, kSwap, kTwo>;
  CUtensorMap mx, mw;
  cudaError_t e = encode(&mx, &mw, o, a, Cfg::kXRows, Cfg::kWRows);
  static bool seen[64];
  if (e == cudaSuccess) e = allow_smem(fp8_split_kernel<BN, kSwap, kTwo>, Cfg::kSmem, seen);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = (unsigned)split;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(tiles * split));
  c.blockDim = dim3(Cfg::kThreads);
  c.dynamicSmemBytes = Cfg::kSmem;
  c.stream = st;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, fp8_split_kernel<BN, kSwap, kTwo>, kSwap ? mw : mx, kSwap ? mx : mw, a, split);
}

cudaError_t launch_fp8_matmul(const void* x, int64_t x_row, const float* xs, int64_t xs_row, int64_t xs_blk,
                              const void* w, int64_t w_row, const float* ws, int64_t ws_row, const void* add,
                              int64_t add_row, void* out, int64_t out_row, int out_f32, int M, int N, int K,
                              cudaStream_t st) {
  int sms = 0;
  cudaError_t e = current_device_sms(&sms);
  if (e != cudaSuccess) return e;
  Fp8Args a = {};
  a.xs = xs;
  a.xs_row = xs_row;
  a.xs_blk = xs_blk;
  a.ws = ws;
  a.ws_row = ws_row;
  a.add = static_cast<const __nv_bfloat16*>(add);
  a.add_row = add_row;
  a.out = out;
  a.out_row = out_row;
  a.out_f32 = out_f32;
  a.M = M;
  a.N = N;
  a.K = K;
  a.vec = ((uintptr_t)out & 15u) == 0 && (out_row * (out_f32 ? 4 : 2)) % 16 == 0 &&
          (!add || (((uintptr_t)add & 15u) == 0 && add_row % 8 == 0));
  const Operands o = {x, w, x_row, w_row};
  // Few tiles: K is split over a cluster until the CTAs fill the GPU, with at
  // least two K blocks each.  Up to 64 tokens the weights' 128 rows lie on
  // the MMA's row side and the tokens (16, 32 or 64) on its column side, two
  // CTAs per SM; past that the tokens take the row side, where a scale
  // thread's activation scale is one value instead of one per column.
  // Measured (us, K x N): M=128 7168 x 4096, tokens on columns 14.5 / on rows
  // 11.9; 2048 x 7168 11.2 / 9.6; M=64, tokens on rows 22.6 against 13.0 and
  // 13.0 against 9.7; M=1 7168 x 4096 split 1 / 2 / 4 / 8: 22.3 / 12.4 / 8.1
  // / 7.8; M=256 4096 x 4096 split 1 / 2 / 4: 18.4 / 12.8 / 18.5 (two waves).
  const int nk = (K + 127) / 128;
  const int bn = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  const int64_t tiles = (int64_t)((M + bn - 1) / bn) * ((N + 127) / 128);
  const int slots = bn == 128 ? sms : 2 * sms;
  if (tiles <= slots / 2) {
    int split = 1;
    while (split < 8 && tiles * split * 2 <= slots && nk >= 4 * split) split *= 2;
    switch (bn) {
      case 16: return launch_split<16, true, true>(o, a, (int)tiles, split, st);
      case 32: return launch_split<32, true, true>(o, a, (int)tiles, split, st);
      case 64: return launch_split<64, true, true>(o, a, (int)tiles, split, st);
      default: return launch_split<128, false, false>(o, a, (int)tiles, split, st);
    }
  }
  // Many tiles: 128 x 256 keeps the tensor cores busier, 128 x 128 leaves
  // less of the last wave idle; a wave of the former takes about 1.25 times
  // as long (M=512 4096 x 4096: 20.6 against 16.8 us, one wave each; M=768
  // 20.8 against 30.6, one and two).
  const int64_t t256 = (int64_t)((M + 127) / 128) * ((N + 255) / 256);
  const int64_t t128 = (int64_t)((M + 127) / 128) * ((N + 127) / 128);
  const int64_t w256 = (t256 + sms - 1) / sms, w128 = (t128 + sms - 1) / sms;
  if (5 * w256 <= 4 * w128) return launch_gemm<256, false>(o, a, sms, st);
  return launch_gemm<128, false>(o, a, sms, st);
}

}  // namespace moe_fp4
