// extern "C" entry points of the operators on a paged cache of 4 bits: its
// step, the norms and the rotation that fill it, what it holds, and attention
// over it.  Argument validation only; the contract of each function is in
// include/moe_fp4.h.
#include <cmath>

#include "attention.cuh"
#include "host.cuh"

using namespace moe_fp4;

namespace {

bool aligned(const void* p, unsigned bytes) { return ((uintptr_t)p & (bytes - 1)) == 0; }
int done(cudaError_t e) { return e == cudaSuccess ? MOE_FP4_OK : report_cuda_error(e); }
bool positive(float v) { return std::isfinite(v) && v > 0.f; }

bool page_ok(int page_size) { return page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128; }
bool dim_ok(int D) { return D == 64 || D == 128 || D == 256; }

// T rows of heads x D bf16 values in 16-byte accesses.  Input rows may repeat
// (strides of 0); `own`: outputs, whose rows and heads must not overlap.
bool heads_ok(const void* p, int64_t row, int64_t head, int T, int heads, int D, bool own) {
  if (!p || !aligned(p, 16) || row % 8 != 0 || head % 8 != 0 || row < 0 || head < 0) return false;
  if (!own) return true;
  if (heads > 1 && head < D) return false;
  if (T <= 1) return true;
  // heads within rows, or rows within heads
  return row >= (int64_t)(heads - 1) * head + D || (row >= D && (heads == 1 || head >= (int64_t)(T - 1) * row + D));
}

}  // namespace

extern "C" {

int moe_fp4_cache_step(const moe_fp4_cache_step_args* p, void* stream) {
  if (!p || p->R < 0 || p->tokens < 0 || p->table_width < 0 || p->free_capacity < 0) return MOE_FP4_EINVAL;
  if (!page_ok(p->page_size) || p->R > 65536) return MOE_FP4_EUNSUPPORTED;
  const moe_fp4_cache_step_args& a = *p;
  if (!a.offsets || !a.free_count || !a.free_count_out) return MOE_FP4_EINVAL;
  if (a.R > 0 && (!a.lengths || !a.new_tokens || !a.lengths_out || !a.accepted)) return MOE_FP4_EINVAL;
  if (a.R > 0 && a.table_width > 0 && (!a.tables || a.table_row < (a.R > 1 ? a.table_width : 0))) return MOE_FP4_EINVAL;
  if (a.free_capacity > 0 && !a.free_pages) return MOE_FP4_EINVAL;
  if (a.tokens > 0 && (!a.positions || !a.slots)) return MOE_FP4_EINVAL;
  for (const void* q : {(const void*)a.lengths, (const void*)a.new_tokens, (const void*)a.tables,
                        (const void*)a.free_pages, (const void*)a.free_count, (const void*)a.offsets,
                        (const void*)a.positions, (const void*)a.lengths_out, (const void*)a.free_count_out,
                        (const void*)a.accepted})
    if (!aligned(q, 4)) return MOE_FP4_EINVAL;
  if (!aligned(a.slots, 8)) return MOE_FP4_EINVAL;
  return done(launch_cache_step(a, static_cast<cudaStream_t>(stream)));
}

int moe_fp4_qk_norm_rope(const moe_fp4_qk_norm_rope_args* p, void* stream) {
  if (!p || p->T < 0 || p->Hq <= 0 || p->Hkv <= 0 || p->D <= 0 || p->rot < 0) return MOE_FP4_EINVAL;
  const moe_fp4_qk_norm_rope_args& a = *p;
  if (!dim_ok(a.D) || a.rot % 16 != 0 || a.rot > a.D || (int64_t)a.Hq + 2 * (int64_t)a.Hkv > 65536)
    return MOE_FP4_EUNSUPPORTED;
  if (!std::isfinite(a.eps) || a.eps < 0.f || !std::isfinite(a.offset)) return MOE_FP4_EINVAL;
  if (a.cache) {
    if (!page_ok(a.page_size)) return MOE_FP4_EUNSUPPORTED;
    if (a.pages <= 0 || !aligned(a.cache, 16) || !positive(a.k_scale) || !positive(a.v_scale)) return MOE_FP4_EINVAL;
  }
  if (a.rotary && (a.rot == 0 || a.positions_max <= 0 || !aligned(a.rotary, 16))) return MOE_FP4_EINVAL;
  if (a.T == 0) return MOE_FP4_OK;
  if (!heads_ok(a.q_in, a.q_row, a.q_head, a.T, a.Hq, a.D, false) ||
      !heads_ok(a.k_in, a.k_row, a.k_head, a.T, a.Hkv, a.D, false) ||
      !heads_ok(a.q_out, a.q_out_row, a.q_out_head, a.T, a.Hq, a.D, true))
    return MOE_FP4_EINVAL;
  if (a.cache) {
    if (!heads_ok(a.v_in, a.v_row, a.v_head, a.T, a.Hkv, a.D, false) || !a.slots || !aligned(a.slots, 8))
      return MOE_FP4_EINVAL;
  } else if (!heads_ok(a.k_out, a.k_out_row, a.k_out_head, a.T, a.Hkv, a.D, true)) {
    return MOE_FP4_EINVAL;
  }
  if (a.rotary && (!a.positions || !aligned(a.positions, a.positions_i64 ? 8 : 4))) return MOE_FP4_EINVAL;
  if (!aligned(a.w_q, 16) || !aligned(a.w_k, 16)) return MOE_FP4_EINVAL;
  return done(launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)));
}

int moe_fp4_cache_read(const void* cache, int pages, int page_size, int Hkv, int D, const int64_t* slots,
                       float k_scale, float v_scale, void* k_out, void* v_out, int T, void* stream) {
  if (T < 0 || Hkv <= 0 || pages <= 0) return MOE_FP4_EINVAL;
  if (!dim_ok(D) || !page_ok(page_size) || Hkv > 65536) return MOE_FP4_EUNSUPPORTED;
  if (!positive(k_scale) || !positive(v_scale)) return MOE_FP4_EINVAL;
  if (T == 0) return MOE_FP4_OK;
  if (!cache || !slots || !k_out || !v_out || !aligned(cache, 16) || !aligned(slots, 8) || !aligned(k_out, 16) ||
      !aligned(v_out, 16))
    return MOE_FP4_EINVAL;
  return done(launch_cache_read(static_cast<const uint8_t*>(cache), (int64_t)pages * page_size, page_size, Hkv, D,
                                slots, k_scale, v_scale, k_out, v_out, T, static_cast<cudaStream_t>(stream)));
}

static int check_attention_sizes(int R, int Hq, int Hkv, int D) {
  if (R < 0 || Hq <= 0 || Hkv <= 0 || D <= 0) return MOE_FP4_EINVAL;
  if (!dim_ok(D) || Hq % Hkv != 0 || Hq / Hkv > 64 || Hq > 65536 || R > 65536) return MOE_FP4_EUNSUPPORTED;
  return MOE_FP4_OK;
}

size_t moe_fp4_attention_workspace_bytes(int R_max, int Hq, int Hkv, int D) {
  return check_attention_sizes(R_max, Hq, Hkv, D) == MOE_FP4_OK ? attention_workspace_bytes(R_max, Hq, Hkv, D) : 0;
}

int moe_fp4_attention(const moe_fp4_attention_args* p, void* stream) {
  if (!p || p->T < 0) return MOE_FP4_EINVAL;
  const moe_fp4_attention_args& a = *p;
  const int st = check_attention_sizes(a.R, a.Hq, a.Hkv, a.D);
  if (st != MOE_FP4_OK) return st;
  if (!page_ok(a.page_size)) return MOE_FP4_EUNSUPPORTED;
  if (a.pages <= 0 || a.table_width < 0 || a.window < 0) return MOE_FP4_EINVAL;
  // (a step past the last token is counted in 32 bits too)
  if ((int64_t)a.table_width * a.page_size > INT32_MAX - 1023 || (int64_t)a.T * a.Hq > INT32_MAX)
    return MOE_FP4_EUNSUPPORTED;
  if (!std::isfinite(a.scale) || !positive(a.k_scale) || !positive(a.v_scale)) return MOE_FP4_EINVAL;
  if (a.T == 0) return MOE_FP4_OK;
  if (!heads_ok(a.q, a.q_row, a.q_head, a.T, a.Hq, a.D, false) ||
      !heads_ok(a.out, a.out_row, a.out_head, a.T, a.Hq, a.D, true))
    return MOE_FP4_EINVAL;
  if (!a.cache || !aligned(a.cache, 16) || !a.offsets || !aligned(a.offsets, 4) || !aligned(a.sinks, 4) ||
      !aligned(a.lse, 4) || !aligned(a.lengths, 4) || !aligned(a.tables, 4))
    return MOE_FP4_EINVAL;
  if (a.R > 0 && (!a.lengths || (a.table_width > 0 && (!a.tables || (a.R > 1 && a.table_row < a.table_width)))))
    return MOE_FP4_EINVAL;
  if (!a.workspace || !aligned(a.workspace, 256) ||
      a.workspace_bytes < attention_workspace_bytes(a.R, a.Hq, a.Hkv, a.D))
    return MOE_FP4_EWORKSPACE;
  return done(launch_attention(a, static_cast<cudaStream_t>(stream)));
}

int moe_fp4_attention_status(uint32_t* flags, int clear, void* stream) {
  if (!flags) return MOE_FP4_EINVAL;
  void* word = nullptr;
  cudaError_t e = attention_status_address(&word);
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

}  // extern "C"
