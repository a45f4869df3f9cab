// Arguments and launchers of the operators around the layer (fp8.cu,
// norm.cu, router.cu), for their entry points in capi_block.cu.
#pragma once

#include "common.cuh"

namespace moe_fp4 {

// `dependent`: launched as its predecessor's dependent (launch_dependent).
cudaError_t launch_fp8_quantize(const void* x, int64_t x_row, const ActParams* act, void* q, int64_t q_row, float* s,
                                int64_t s_row, int64_t s_blk, int M, int K, bool dependent, cudaStream_t st);
// A product's weight scales, addend, output and sizes.
struct Fp8Product {
  const float* ws;
  int64_t ws_row;
  const void* add;
  int64_t add_row;
  void* out;
  int64_t out_row;
  int out_f32;
  int M, N, K;
};
// `after_quantizer`: the stream's last launch is launch_fp8_quantize of x, in
// plain order.
cudaError_t launch_fp8_matmul(const void* x, int64_t x_row, const float* xs, int64_t xs_row, int64_t xs_blk,
                              const void* w, int64_t w_row, Fp8Product p, bool after_quantizer, cudaStream_t st);
// BF16 x, where fp8_linear_is_fused(M, K).
bool fp8_linear_is_fused(int M, int K);
cudaError_t launch_fp8_linear_fused(const void* x, int64_t x_row, const void* w, int64_t w_row, Fp8Product p,
                                    cudaStream_t st);
cudaError_t fp8_status_address(void** p);

struct NormArgs {
  const void* r;  // residual [M][H], bf16 or f32
  int64_t r_row;
  const uint16_t* b;  // block output [M][H] bf16, or null
  int64_t b_row;
  const void* w_post;  // [H] or null
  const void* w_pre;   // [H] or null (no n)
  int w_f32;
  const void* gate;  // null, or gate[m * g_row + h * g_col]
  int64_t g_row, g_col;
  int g_f32;
  float scale, eps, offset;
  void* r_out;  // residual's type, or null
  int64_t ro_row;
  uint16_t* n;  // bf16, or null
  int64_t n_row;
  uint8_t* q;  // e4m3, or null
  int64_t q_row;
  float* s;
  int64_t s_row, s_blk;
  int M, H;
  int layout, shift, shift_row, staged;  // launch_block_norm's choice
};
// `packed`: every row of every array starts 16-byte aligned and H % 8 == 0.
cudaError_t launch_block_norm(NormArgs a, int res_f32, bool packed, cudaStream_t st);

struct RouteArgs {
  const void* logits;
  int64_t row;
  int f32;
  const float* bias;  // [E] or null
  int sigmoid, renormalize;
  float scale;
  int32_t* ids;
  float* weights;
  int M, E, k;
};
cudaError_t launch_route_topk(const RouteArgs& a, cudaStream_t st);

}  // namespace moe_fp4
