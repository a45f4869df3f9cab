// FP8 products with a scale per block of 128 (moe_fp4_fp8_*): the activation
// quantiser and the launches of the product kernels of gemm_fp8.cuh.
#include "block.cuh"
#include "fp8_quant.cuh"
#include "gemm_fp8.cuh"
#include "host.cuh"

namespace moe_fp4 {

// Status word of the product kernels' bounded waits (moe_fp4_fp8_status).
static __device__ uint32_t g_fp8_status;

cudaError_t fp8_status_address(void** p) { return cudaGetSymbolAddress(p, g_fp8_status); }

// ---------------------------------------------------------------- quantiser
// Per row and 128 columns: s = max|v| / 448 (1 where that is zero), q =
// e4m3_rn(v / s), each step an IEEE FP32 operation; v is the input, or
// act(gate) * up of a gated row [gate | up].  A warp takes 1024 columns of a
// row (512 of a gated one), all its loads under way before the first block's
// maximum.  Sixteen columns a lane halve what is paid per lane and block (the
// scale, its reciprocal, the shuffles) against eight: 16384 x 7168 51.5 us
// against 61.8.
//
// Bound: HBM (that size: 6.9 TB/s of a copy's 6.8; 4096 x 7168 14.8 us, 6.0
// TB/s), with SiLU the instructions of its exact exponential, reciprocal and
// quotients (16384 x 7168 122 us, 4.8 TB/s; with IEEE divisions 139; GELU 128,
// SwiGLU-OAI 140); up to a few hundred rows the launch (64 x 7168 1.7 us, 64 x
// 2048 with SiLU or GELU 2.0, with SwiGLU-OAI 2.4).

// SiLU(g) u in full FP32 precision (the scale of a block follows its largest
// product, and an element near the middle of two E4M3 values turns on it), on
// the V gates and ups of a lane.
template <int V>
__device__ __forceinline__ void silu_gated(const uint4 (&g_raw)[V / 8], const float (&up)[V], float (&v)[V]) {
  // Without a division where 1 + e^-g is below 2^126 and g finite.  (A g below
  // 2^-25 has the divisor 2 exactly, so no remainder is too small.)
  __nv_bfloat162 most;
#pragma unroll
  for (int i = 0; i < V / 8; ++i) {
    const uint32_t p[4] = {g_raw[i].x, g_raw[i].y, g_raw[i].z, g_raw[i].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const __nv_bfloat162 b = __habs2(*reinterpret_cast<const __nv_bfloat162*>(&p[j]));
      most = i + j ? __hmax2(most, b) : b;
    }
  }
  if (fmaxf(__low2float(most), __high2float(most)) < 80.f) {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 g = make_float2(v[2 * i], v[2 * i + 1]);
      const float2 e = make_float2(expf(-g.x), expf(-g.y));
      const float2 x_neg = ffma2(e, both(-1.f), both(-1.f));
      const float2 q = fmul2(quotients(g, x_neg, reciprocals(x_neg)), make_float2(up[2 * i], up[2 * i + 1]));
      v[2 * i] = q.x;
      v[2 * i + 1] = q.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = __fdiv_rn(v[i], 1.0f + expf(-v[i])) * up[i];
  }
}

// min and max that hand a NaN on (fminf and fmaxf take the other operand).
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// SwiGLU-OAI of one gate and up (gated_act's formula), where a NaN stays: the
// block's FP8 form would hide one that the limits had replaced.  The hardware's
// exponential: its error grows with |alpha g| as that of the rounded product
// alpha g does, and is about twice it (expf: 16384 x 7168 150 us for 140).
__device__ __forceinline__ float swiglu_oai(float gate, float up, const ActParams& p) {
  const float g = min_nan(gate, p.limit);
  const float u = min_nan(max_nan(up, -p.limit), p.limit);
  return (u + p.beta) * g / (1.0f + __expf(-p.alpha * g));
}

// A lane takes V consecutive columns (8 or 16) of each of kChunks chunks.  (No
// __restrict__: it would let the compiler read x as data that no kernel
// writes, even before pdl_wait, while the launch before may still write it.)
template <bool kGated, int V, int kChunks>
__global__ void __launch_bounds__(256) fp8_quantize_kernel(const uint16_t* x, int64_t x_row, ActParams act, uint8_t* q,
                                                           int64_t q_row, float* s, int64_t s_row, int64_t s_blk,
                                                           int M, int K) {
  constexpr int kCols = 32 * V;
  pdl_wait();
  pdl_launch_dependents();
  const unsigned groups = (unsigned)(K + kCols * kChunks - 1) / (kCols * kChunks);
  const unsigned task = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  const unsigned m = task / groups;
  if (m >= (unsigned)M) return;
  const int lane = threadIdx.x & 31;
  const int k0 = (int)(task % groups) * (kCols * kChunks) + lane * V;
  const uint16_t* row = x + m * x_row;
  uint4 raw[kChunks][V / 8], raw_up[kChunks][V / 8];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int k = k0 + i * kCols;  // (K % 16 == 0: a lane's columns are there or not)
#pragma unroll
    for (int j = 0; j < V / 8; ++j) {
      raw[i][j] = raw_up[i][j] = make_uint4(0, 0, 0, 0);
      if (k < K) {
        raw[i][j] = *reinterpret_cast<const uint4*>(row + k + 8 * j);
        if (kGated) raw_up[i][j] = *reinterpret_cast<const uint4*>(row + K + k + 8 * j);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int k = k0 + i * kCols;
    float v[V];
#pragma unroll
    for (int j = 0; j < V / 8; ++j) bf16x8_to_float(raw[i][j], v + 8 * j);
    if (kGated) {
      float up[V];
#pragma unroll
      for (int j = 0; j < V / 8; ++j) bf16x8_to_float(raw_up[i][j], up + 8 * j);
      if (act.kind == MOE_FP4_ACT_SILU) {
        silu_gated<V>(raw[i], up, v);
      } else if (act.kind == MOE_FP4_ACT_SWIGLUOAI) {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = swiglu_oai(v[j], up[j], act);
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = gated_act(v[j], up[j], act);
      }
    }
    const float sc = block_scale(block_amax(v));
    if (k < K) {
      uint32_t w[V / 4];
      e4m3_quotients(v, sc, w);
      uint8_t* to = q + m * q_row + k;
      if constexpr (V == 16)
        *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
      else
        *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
      if (lane % (128 / V) == 0) s[m * s_row + (int64_t)(k / 128) * s_blk] = sc;
    }
  }
}

template <bool kGated, int V, int kChunks>
static cudaError_t launch_quantize(const void* x, int64_t x_row, const ActParams& act, void* q, int64_t q_row, float* s,
                                   int64_t s_row, int64_t s_blk, int M, int K, unsigned warps, bool dependent,
                                   cudaStream_t st) {
  // (tasks fit 32 bits: each stands for 16 values or a whole row in memory)
  const int64_t tasks = (int64_t)M * ((K + 32 * V * kChunks - 1) / (32 * V * kChunks));
  const unsigned grid = (unsigned)((tasks + warps - 1) / warps);
  const uint16_t* xp = static_cast<const uint16_t*>(x);
  uint8_t* qp = static_cast<uint8_t*>(q);
  return launch_smem(fp8_quantize_kernel<kGated, V, kChunks>, grid, 32 * warps, 0, dependent, st, xp, x_row, act, qp,
                     q_row, s, s_row, s_blk, M, K);
}

cudaError_t launch_fp8_quantize(const void* x, int64_t x_row, const ActParams* act, void* q, int64_t q_row, float* s,
                                int64_t s_row, int64_t s_blk, int M, int K, bool dependent, cudaStream_t st) {
  int sms = 0;
  const cudaError_t e = current_device_sms(&sms);
  if (e != cudaSuccess) return e;
  const ActParams none = {MOE_FP4_ACT_SILU, 0.f, 0.f, 0.f};
  // 1024 columns per warp where that gives every SM its warps (with SiLU 512:
  // 16384 x 7168 122 us against 128 with 1024 at fewer warps per SM), else
  // 256, so that a few rows spread over the GPU
  const bool few = (int64_t)M * ((K + 1023) / 1024) < 16 * sms;
  if (act && few)
    return launch_quantize<true, 8, 1>(x, x_row, *act, q, q_row, s, s_row, s_blk, M, K, 4, dependent, st);
  if (act) return launch_quantize<true, 16, 1>(x, x_row, *act, q, q_row, s, s_row, s_blk, M, K, 8, dependent, st);
  if (few) return launch_quantize<false, 8, 1>(x, x_row, none, q, q_row, s, s_row, s_blk, M, K, 4, dependent, st);
  return launch_quantize<false, 16, 2>(x, x_row, none, q, q_row, s, s_row, s_blk, M, K, 8, dependent, st);
}

// ------------------------------------------------------------------ product
template <int BN>
__global__ void __launch_bounds__(F8Cfg<BN, false>::kThreads, 1)
    fp8_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                     const __grid_constant__ Fp8Args a) {
  gemm_fp8_persistent<BN, false>(&map_a, &map_b, a, &g_fp8_status);
}

template <int BN, bool kSwap, bool kTwo>
__global__ void __launch_bounds__(F8Cfg<BN, kSwap, kTwo>::kThreads, kTwo ? 2 : 1)
    fp8_split_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                     const __grid_constant__ Fp8Args a,
                     int split) {
  gemm_fp8_persistent<BN, kSwap, kTwo, true>(&map_a, &map_b, a, &g_fp8_status, split);
}

// The same for at most eight BF16 tokens (a.xb), quantised by the kernel.
template <int kXq>
__global__ void __launch_bounds__(F8Cfg<16, true, true, kXq>::kThreads, 2)
    fp8_linear_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ Fp8Args a, int split) {
  gemm_fp8_persistent<16, true, true, true, kXq>(&map_w, &map_w, a, &g_fp8_status, split);
}

// The product kernels' arguments but for the activations.
static Fp8Args args_of(const Fp8Product& p) {
  Fp8Args a = {};
  a.ws = p.ws;
  a.ws_row = p.ws_row;
  a.add = static_cast<const __nv_bfloat16*>(p.add);
  a.add_row = p.add_row;
  a.out = p.out;
  a.out_row = p.out_row;
  a.out_f32 = p.out_f32;
  a.M = p.M;
  a.N = p.N;
  a.K = p.K;
  a.vec = ((uintptr_t)p.out & 15u) == 0 && (p.out_row * (p.out_f32 ? 4 : 2)) % 16 == 0 &&
          (!p.add || (((uintptr_t)p.add & 15u) == 0 && p.add_row % 8 == 0));
  a.pairs = ((uintptr_t)p.out % (p.out_f32 ? 8 : 4)) == 0 && p.out_row % 2 == 0;
  if (a.vec && ((uintptr_t)p.out & 31u) == 0 && (p.out_row * (p.out_f32 ? 4 : 2)) % 32 == 0) a.vec = 2;
  return a;
}

struct Operands {
  const void *x, *w;
  int64_t x_row, w_row;
};

// Launch with a cluster of `split` CTAs, as a dependent of the launch before
// (see launch_dependent).  Behind our own quantiser (a.early) the first
// weight loads, too, run beside it, before the wait: the quantiser is then
// launched in plain stream order, so whatever wrote the weights has finished.
template <class Kern, class... Args>
static cudaError_t launch_product(Kern kern, int64_t ctas, int threads, size_t smem, int split,
                                  cudaStream_t st, const Args&... args) {
  cudaLaunchAttribute at[2];
  unsigned n = 0;
  if (split > 1) {
    at[n].id = cudaLaunchAttributeClusterDimension;
    at[n].val.clusterDim.x = (unsigned)split;
    at[n].val.clusterDim.y = at[n].val.clusterDim.z = 1;
    ++n;
  }
  at[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)ctas);
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = at;
  c.numAttrs = n;
  return cudaLaunchKernelEx(&c, kern, args...);
}

static cudaError_t encode(CUtensorMap* mx, CUtensorMap* mw, const Operands& o, const Fp8Args& a, int x_rows,
                          int w_rows) {
  CUresult r = encode_u8_map_2d(mx, o.x, (uint64_t)a.K, (uint64_t)a.M, (uint64_t)o.x_row, (uint32_t)x_rows);
  if (r == CUDA_SUCCESS)
    r = encode_u8_map_2d(mw, o.w, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)o.w_row, (uint32_t)w_rows);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int BN>
static cudaError_t launch_gemm(const Operands& o, const Fp8Args& a, int sms, cudaStream_t st) {
  using Cfg = F8Cfg<BN, false>;
  CUtensorMap mx, mw;
  cudaError_t e = encode(&mx, &mw, o, a, Cfg::kXRows, Cfg::kWRows);
  static bool seen[64];
  if (e == cudaSuccess) e = allow_smem(fp8_gemm_kernel<BN>, Cfg::kSmem, seen);
  if (e != cudaSuccess) return e;
  const int64_t tiles =
      (int64_t)((a.M + Cfg::kXRows - 1) / Cfg::kXRows) * ((a.N + Cfg::kWRows - 1) / Cfg::kWRows);
  return launch_product(fp8_gemm_kernel<BN>, tiles < sms ? tiles : sms, Cfg::kThreads, Cfg::kSmem, 1, st,
                        mx, mw, a);
}

template <int BN, bool kSwap, bool kTwo>
static cudaError_t launch_split(const Operands& o, const Fp8Args& a, int tiles, int split, cudaStream_t st) {
  using Cfg = F8Cfg<BN, kSwap, kTwo>;
  CUtensorMap mx, mw;
  cudaError_t e = encode(&mx, &mw, o, a, Cfg::kXRows, Cfg::kWRows);
  static bool seen[64];
  if (e == cudaSuccess) e = allow_smem(fp8_split_kernel<BN, kSwap, kTwo>, Cfg::kSmem, seen);
  if (e != cudaSuccess) return e;
  return launch_product(fp8_split_kernel<BN, kSwap, kTwo>, (int64_t)tiles * split, Cfg::kThreads, Cfg::kSmem, split, st,
                        kSwap ? mw : mx, kSwap ? mx : mw, a, split);
}

// Few tiles: K is split over a cluster until the CTAs fill `slots`, with at
// least two K blocks each.  Up to 16 tokens a CTA has at most 16 blocks
// where eight CTAs can manage that: the kernel that quantises its own tokens
// holds as many (it shares this rule, so that its results are the same).
static int k_split(int64_t tiles, int slots, int nk, int bn) {
  int split = 1;
  while (split < 8 && nk >= 4 * split && (tiles * split * 2 <= slots || (bn == 16 && nk > 16 * split && nk <= 128)))
    split *= 2;
  return split;
}

// The decode band (M <= MOE_FP4_DECODE_MAX_M) with K <= 16384: one launch, no
// workspace (K x N 7168 x 4096, one launch against quantiser and product, in a
// graph: M=1 8.0 / 9.2 us, M=8 9.2 / 9.4 with the weights in L2, 8.9 / 11.4 and
// 9.7 / 11.7 with weights from memory; and one launch less for the host, about
// 3 us of an eager call).
bool fp8_linear_is_fused(int M, int K) { return M <= MOE_FP4_DECODE_MAX_M && K <= 128 * 128; }

template <int kXq>
static cudaError_t launch_fused(const CUtensorMap& mw, const Fp8Args& a, int64_t tiles, int split, cudaStream_t st) {
  using Cfg = F8Cfg<16, true, true, kXq>;
  static bool seen[64];
  const cudaError_t e = allow_smem(fp8_linear_kernel<kXq>, Cfg::kSmem, seen);
  if (e != cudaSuccess) return e;
  return launch_product(fp8_linear_kernel<kXq>, tiles * split, Cfg::kThreads, Cfg::kSmem, split, st, mw, a, split);
}

cudaError_t launch_fp8_linear_fused(const void* x, int64_t x_row, const void* w, int64_t w_row, Fp8Product p,
                                    cudaStream_t st) {
  int sms = 0;
  cudaError_t e = current_device_sms(&sms);
  if (e != cudaSuccess) return e;
  Fp8Args a = args_of(p);
  a.xb = static_cast<const uint16_t*>(x);
  a.xb_row = x_row;
  CUtensorMap mw;
  if (encode_u8_map_2d(&mw, w, (uint64_t)a.K, (uint64_t)a.N, (uint64_t)w_row, kF8BM) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const int64_t tiles = (a.N + 127) / 128;
  const int nk = (a.K + 127) / 128;
  int split = k_split(tiles, 2 * sms, nk, 16);
  if ((nk + split - 1) / split <= 8) return launch_fused<8>(mw, a, tiles, split, st);
  return launch_fused<16>(mw, a, tiles, split, st);
}

cudaError_t launch_fp8_matmul(const void* x, int64_t x_row, const float* xs, int64_t xs_row, int64_t xs_blk,
                              const void* w, int64_t w_row, Fp8Product p, bool after_quantizer, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = current_device_sms(&sms);
  if (e != cudaSuccess) return e;
  Fp8Args a = args_of(p);
  a.xs = xs;
  a.xs_row = xs_row;
  a.xs_blk = xs_blk;
  const int M = p.M, N = p.N, K = p.K;
  const Operands o = {x, w, x_row, w_row};
  a.early = after_quantizer;
  a.xs_vec = xs_row == 1 && xs_blk % 4 == 0 && ((uintptr_t)xs & 15u) == 0 && (M % 4 == 0 || after_quantizer);
  // Up to 32 tokens the weights' 128 rows lie on the MMA's row side and the
  // tokens (16 or 32) on its column side, two CTAs per SM; past that the
  // tokens take the row side, where a scale thread's activation scale is one
  // value instead of one per column.  Measured (us, K x N, weights in L2): 7168 x
  // 4096, M=64 tokens on 64 columns 12.4, on rows 10.4, M=128 14.5 and 11.3;
  // split 1 / 2 / 4 / 8: M=1 7168 x 4096 15.5 / 9.8 / 6.9 / 7.0, M=128 21.3 /
  // 14.6 / 11.1 / 26.7, M=256 4096 x 4096 14.6 / 11.2 / 17.3 / 38.9; with weights
  // from memory 15.9 / 10.5 / 8.9 / 8.8, 21.6 / 15.0 / 12.2 / 28.8 and 15.1 / 11.9
  // / 18.4 / 40.5.
  const int nk = (K + 127) / 128;
  const int bn = M <= 16 ? 16 : M <= 32 ? 32 : 128;
  const int64_t tiles = (int64_t)((M + bn - 1) / bn) * ((N + 127) / 128);
  const int slots = bn == 128 ? sms : 2 * sms;
  // (128 tokens on rows, a CTA's partial sums 64 KB: from 16 K blocks on, M=300
  // 1024 x 1024, eight blocks, split 1 / 2 / 4 6.7 / 7.8 / 7.1 us, M=64 2048 x
  // 7168, sixteen, split 1 / 2 9.6 / 8.5; but always where rows allow no vector
  // stores, which that kernel's last step does not need: M=226 1328 x 999 9.1
  // us in all, 14.4 without.)
  if (bn == 16 || (tiles <= slots / 2 && (bn < 128 || nk >= 16 || !a.vec))) {
    const int split = k_split(tiles, slots, nk, bn);
    switch (bn) {
      case 16: return launch_split<16, true, true>(o, a, (int)tiles, split, st);
      case 32: return launch_split<32, true, true>(o, a, (int)tiles, split, st);
      default: return launch_split<128, false, false>(o, a, (int)tiles, split, st);
    }
  }
  // Many tiles: 128 x 256 takes in less per product, 128 x 128 leaves less of
  // the last wave idle; a wave of the former takes 1.2 to 1.4 times as long
  // (256 against 128 wide: M=512 4096 x 4096, one wave each, 17.1 against 14.0
  // us; M=768, one and two, 17.8 against 24.3; M=700 7168 x 7168, two and
  // three, 51.1 against 56.9; M=4096 7168 x 4096, four and seven, 97 against
  // 124).  K split in clusters for the tiles of the last wave, or for 256-wide
  // tiles, gained at none of these but M=700: a cluster's sums pass through
  // shared memory at some 15 bytes a cycle and SM.
  const int64_t t256 = (int64_t)((M + 127) / 128) * ((N + 255) / 256);
  const int64_t t128 = (int64_t)((M + 127) / 128) * ((N + 127) / 128);
  const int64_t w256 = (t256 + sms - 1) / sms, w128 = (t128 + sms - 1) / sms;
  if (4 * w256 <= 3 * w128) return launch_gemm<256>(o, a, sms, st);
  return launch_gemm<128>(o, a, sms, st);
}

}  // namespace moe_fp4
