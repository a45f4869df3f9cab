// extern "C" entry points of the operators around the layer: the FP8 product
// and its activation quantiser, the norms around a block, the router's
// choice.  Argument validation only; the contract of each function is in
// include/moe_fp4.h.
#include <cmath>

#include "block.cuh"
#include "host.cuh"

using namespace moe_fp4;

namespace {

bool aligned(const void* p, unsigned bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }
int done(cudaError_t e) { return e == cudaSuccess ? MOE_FP4_OK : report_cuda_error(e); }
size_t align256(size_t b) { return (b + 255) & ~(size_t)255; }
int64_t blocks128(int64_t n) { return (n + 127) / 128; }

// M x cols elements with a row stride: the rows must not overlap.
bool rows_ok(int64_t row, int64_t cols, int M) { return row >= cols || M == 1; }

int check_fp8_sizes(int M, int N, int K) {
  if (M < 0 || N <= 0 || K <= 0) return MOE_FP4_EINVAL;
  if (K % 16 != 0) return MOE_FP4_EUNSUPPORTED;
  // tile indices and tensor-map coordinates are 32-bit
  if (blocks128(M) * blocks128(N) * 8 > (int64_t)INT32_MAX || K > (1 << 30) || N > (1 << 30) || M > (1 << 30))
    return MOE_FP4_EUNSUPPORTED;
  return MOE_FP4_OK;
}

int check_fp8_operands(const void* x, int64_t x_row, const void* w, int64_t w_row, const float* w_s, int64_t ws_row,
                       const void* add, int64_t add_row, const void* out, int64_t out_row, int out_f32, int M, int N,
                       int K) {
  if (!x || !w || !w_s || !out || (out_f32 != 0 && out_f32 != 1)) return MOE_FP4_EINVAL;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(w_s, 4) || !aligned(out, out_f32 ? 4 : 2) || !aligned(add, 2))
    return MOE_FP4_EINVAL;
  if (!rows_ok(x_row, K, M) || !rows_ok(w_row, K, N) || w_row % 16 != 0 || !rows_ok(ws_row, blocks128(K), (int)blocks128(N)) ||
      !rows_ok(out_row, N, M) || (add && !rows_ok(add_row, N, M)))
    return MOE_FP4_EINVAL;
  return MOE_FP4_OK;
}

}  // namespace

extern "C" {

int moe_fp4_fp8_quantize(const void* x_bf16, int64_t x_row, const moe_fp4_activation* act, void* q, int64_t q_row,
                         float* s, int64_t s_row, int64_t s_block, int M, int K, void* stream) {
  const int st = check_fp8_sizes(M, 1, K);
  if (st != MOE_FP4_OK) return st;
  ActParams ap = {MOE_FP4_ACT_SILU, 0.f, 0.f, 0.f};
  if (act) {
    if (act->kind != MOE_FP4_ACT_SILU && act->kind != MOE_FP4_ACT_GELU_TANH && act->kind != MOE_FP4_ACT_SWIGLUOAI)
      return MOE_FP4_EINVAL;
    if (act->kind == MOE_FP4_ACT_SWIGLUOAI &&
        (!std::isfinite(act->alpha) || !std::isfinite(act->beta) || !(act->limit > 0.f)))
      return MOE_FP4_EINVAL;
    ap = {act->kind, act->alpha, act->beta, act->limit};
  }
  if (M == 0) return MOE_FP4_OK;
  if (!x_bf16 || !q || !s || !aligned(x_bf16, 16) || !aligned(q, 16) || !aligned(s, 4)) return MOE_FP4_EINVAL;
  if (!rows_ok(x_row, act ? 2 * (int64_t)K : K, M) || !rows_ok(q_row, K, M) || x_row % 8 != 0 || q_row % 16 != 0)
    return MOE_FP4_EINVAL;
  if (s_row < 0 || s_block < 0) return MOE_FP4_EINVAL;
  return done(launch_fp8_quantize(x_bf16, x_row, act ? &ap : nullptr, q, q_row, s, s_row, s_block, M, K, true,
                                  static_cast<cudaStream_t>(stream)));
}

int moe_fp4_fp8_matmul(const void* x_q, int64_t x_row, const float* x_s, int64_t xs_row, int64_t xs_block,
                       const void* w, int64_t w_row, const float* w_s, int64_t ws_row, const void* add_bf16,
                       int64_t add_row, void* out, int64_t out_row, int out_f32, int M, int N, int K, void* stream) {
  int st = check_fp8_sizes(M, N, K);
  if (st != MOE_FP4_OK) return st;
  if (M == 0) return MOE_FP4_OK;
  st = check_fp8_operands(x_q, x_row, w, w_row, w_s, ws_row, add_bf16, add_row, out, out_row, out_f32, M, N, K);
  if (st != MOE_FP4_OK) return st;
  if (!x_s || !aligned(x_s, 4) || x_row % 16 != 0 || xs_row < 0 || xs_block < 0) return MOE_FP4_EINVAL;
  const Fp8Product p = {w_s, ws_row, add_bf16, add_row, out, out_row, out_f32, M, N, K};
  return done(launch_fp8_matmul(x_q, x_row, x_s, xs_row, xs_block, w, w_row, p, false,
                                static_cast<cudaStream_t>(stream)));
}

// Rows of a K block's scales in the workspace: whole 16 bytes of them.
static size_t scale_rows(size_t M) { return (M + 3) / 4 * 4; }

size_t moe_fp4_fp8_linear_workspace_bytes(int M_max, int K) {
  if (check_fp8_sizes(M_max, 1, K) != MOE_FP4_OK) return 0;
  const size_t M = M_max < 1 ? 1 : (size_t)M_max;
  return align256(M * K) + align256(scale_rows(M) * blocks128(K) * sizeof(float));
}

int moe_fp4_fp8_linear(const void* x_bf16, int64_t x_row, const void* w, int64_t w_row, const float* w_s,
                       int64_t ws_row, const void* add_bf16, int64_t add_row, void* out, int64_t out_row, int out_f32,
                       int M, int N, int K, void* workspace, size_t workspace_bytes, void* stream) {
  int st = check_fp8_sizes(M, N, K);
  if (st != MOE_FP4_OK) return st;
  if (M == 0) return MOE_FP4_OK;
  st = check_fp8_operands(x_bf16, x_row, w, w_row, w_s, ws_row, add_bf16, add_row, out, out_row, out_f32, M, N, K);
  if (st != MOE_FP4_OK) return st;
  if (x_row % 8 != 0) return MOE_FP4_EINVAL;
  const bool fused = fp8_linear_is_fused(M, K);
  if (!workspace && !fused) return MOE_FP4_EWORKSPACE;
  if (workspace && (!aligned(workspace, 256) || workspace_bytes < moe_fp4_fp8_linear_workspace_bytes(M, K)))
    return MOE_FP4_EWORKSPACE;
  const Fp8Product p = {w_s, ws_row, add_bf16, add_row, out, out_row, out_f32, M, N, K};
  if (fused) return done(launch_fp8_linear_fused(x_bf16, x_row, w, w_row, p, static_cast<cudaStream_t>(stream)));
  float* s = reinterpret_cast<float*>(static_cast<char*>(workspace) + align256((size_t)M * K));
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const int64_t block = (int64_t)scale_rows((size_t)M);
  const cudaError_t e = launch_fp8_quantize(x_bf16, x_row, nullptr, workspace, K, s, 1, block, M, K, false, cs);
  if (e != cudaSuccess) return report_cuda_error(e);
  return done(launch_fp8_matmul(workspace, K, s, 1, block, w, w_row, p, true, cs));
}

int moe_fp4_fp8_status(uint32_t* flags, int clear, void* stream) {
  if (!flags) return MOE_FP4_EINVAL;
  void* word = nullptr;
  cudaError_t e = fp8_status_address(&word);
  uint32_t v = 0;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&v, word, sizeof(v), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && clear) e = cudaMemsetAsync(word, 0, sizeof(v), s);
  if (e == cudaSuccess && clear) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return report_cuda_error(e);
  *flags = v;
  return MOE_FP4_OK;
}

int moe_fp4_block_norm(const moe_fp4_block_norm_args* p, void* stream) {
  if (!p || p->M < 0 || p->H <= 0) return MOE_FP4_EINVAL;
  if (p->H > 32768) return MOE_FP4_EUNSUPPORTED;
  if (!std::isfinite(p->scale) || !std::isfinite(p->offset) || !std::isfinite(p->eps) || p->eps < 0.f)
    return MOE_FP4_EINVAL;
  if (p->q && p->H % 16 != 0) return MOE_FP4_EUNSUPPORTED;
  if (p->M == 0) return MOE_FP4_OK;
  const int M = p->M, H = p->H;
  if (!p->residual || (p->w_pre && !p->normed && !p->q) || ((p->normed || p->q) && !p->w_pre)) return MOE_FP4_EINVAL;
  if (!p->residual_out && !p->w_pre) return MOE_FP4_EINVAL;  // nothing to compute
  if (p->q && !p->s) return MOE_FP4_EINVAL;
  const bool gated = p->block_out && p->gate;
  if (gated && (p->gate_row < 0 || (p->gate_col != 0 && p->gate_col != 1))) return MOE_FP4_EINVAL;
  const unsigned rb = p->residual_f32 ? 4 : 2, wb = p->weights_f32 ? 4 : 2, gb = p->gate_f32 ? 4 : 2;
  if (!aligned(p->residual, rb) || !aligned(p->residual_out, rb) || !aligned(p->block_out, 2) ||
      !aligned(p->w_post, wb) || !aligned(p->w_pre, wb) || !aligned(p->normed, 2) || !aligned(p->s, 4) ||
      (gated && !aligned(p->gate, gb)))
    return MOE_FP4_EINVAL;
  // (input rows may repeat: a stride of 0 reads one row for every token)
  if (p->residual_row < 0 || p->block_row < 0 || (p->residual_out && !rows_ok(p->residual_out_row, H, M)) ||
      (p->normed && !rows_ok(p->normed_row, H, M)) || (p->q && !rows_ok(p->q_row, H, M)) || p->s_row < 0 ||
      p->s_block < 0)
    return MOE_FP4_EINVAL;
  auto vec = [&](const void* q, int64_t row, unsigned bytes) {
    return !q || (aligned(q, 16) && (row * bytes) % 16 == 0);
  };
  const bool v = H % 8 == 0 && vec(p->residual, p->residual_row, rb) && vec(p->residual_out, p->residual_out_row, rb) &&
                 vec(p->block_out, p->block_row, 2) && vec(p->w_post, 0, wb) && vec(p->w_pre, 0, wb) &&
                 vec(p->normed, p->normed_row, 2) && vec(p->q, p->q_row, 1) &&
                 (!gated || p->gate_col == 0 || vec(p->gate, p->gate_row, gb));
  if (p->q && !v) return MOE_FP4_EINVAL;
  NormArgs a = {};
  a.r = p->residual;
  a.r_row = p->residual_row;
  a.b = static_cast<const uint16_t*>(p->block_out);
  a.b_row = p->block_row;
  a.w_post = p->block_out ? p->w_post : nullptr;
  a.w_pre = p->w_pre;
  a.w_f32 = p->weights_f32;
  a.gate = gated ? p->gate : nullptr;
  a.g_row = p->gate_row;
  a.g_col = p->gate_col;
  a.g_f32 = p->gate_f32;
  a.scale = p->scale;
  a.eps = p->eps;
  a.offset = p->offset;
  a.r_out = p->residual_out;
  a.ro_row = p->residual_out_row;
  a.n = static_cast<uint16_t*>(p->normed);
  a.n_row = p->normed_row;
  a.q = static_cast<uint8_t*>(p->q);
  a.q_row = p->q_row;
  a.s = p->s;
  a.s_row = p->s_row;
  a.s_blk = p->s_block;
  a.M = M;
  a.H = H;
  return done(launch_block_norm(a, p->residual_f32 ? 1 : 0, v, static_cast<cudaStream_t>(stream)));
}

int moe_fp4_route_topk(const void* logits, int64_t logits_row, int logits_f32, const float* bias, int score,
                       int renormalize, float scale, int32_t* topk_ids, float* topk_weights, int M, int E, int top_k,
                       void* stream) {
  if (M < 0 || E <= 0 || top_k <= 0 || (score != MOE_FP4_SCORE_SOFTMAX && score != MOE_FP4_SCORE_SIGMOID))
    return MOE_FP4_EINVAL;
  if (top_k > 16 || top_k > E || E > 65536) return MOE_FP4_EUNSUPPORTED;
  if ((bias && score != MOE_FP4_SCORE_SIGMOID) || !std::isfinite(scale)) return MOE_FP4_EINVAL;
  if (M == 0) return MOE_FP4_OK;
  if (!logits || !topk_ids || !topk_weights || logits_row < 0) return MOE_FP4_EINVAL;
  if (!aligned(logits, logits_f32 ? 4 : 2) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4))
    return MOE_FP4_EINVAL;
  RouteArgs a = {logits, logits_row, logits_f32, bias,         score == MOE_FP4_SCORE_SIGMOID, renormalize,
                 scale,  topk_ids,   topk_weights, M,          E,                              top_k};
  return done(launch_route_topk(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
