// Arguments and launchers of the operators on a paged cache of 4 bits
// (cache.cu, rope.cu, attention.cu), for their entry points in
// capi_attention.cu, and the cache's layout.
#pragma once

#include "common.cuh"

namespace moe_fp4 {

// Of each 16 tokens of a head: their keys, then their values, each 16 rows of
// D / 2 bytes (E2M1) and 16 rows of D / 16 scales (E4M3).
constexpr int kCacheBlock = 16;
__host__ __device__ constexpr int cache_half_bytes(int D) { return 9 * D; }
__host__ __device__ constexpr int cache_block_bytes(int D) { return 18 * D; }

// Where a token's key lies: the bytes of its codes and of its scales (its
// value: cache_half_bytes further).
struct CachePlace {
  int64_t codes, scales;
};
__device__ __forceinline__ CachePlace cache_place(int64_t slot, int head, int Hkv, int page_size, int D) {
  const int64_t page = slot / page_size;
  const int in = (int)(slot - page * page_size), row = in % kCacheBlock;
  const int64_t block = (page * Hkv + head) * (page_size / kCacheBlock) + in / kCacheBlock;
  const int64_t at = block * cache_block_bytes(D);
  return {at + row * (D / 2), at + 8 * D + row * (D / 16)};
}

cudaError_t launch_cache_step(const moe_fp4_cache_step_args& a, cudaStream_t st);
cudaError_t launch_qk_norm_rope(const moe_fp4_qk_norm_rope_args& a, cudaStream_t st);
cudaError_t launch_cache_read(const uint8_t* cache, int64_t slots_max, int page_size, int Hkv, int D,
                              const int64_t* slots, float k_scale, float v_scale, void* k_out, void* v_out, int T,
                              cudaStream_t st);
size_t attention_workspace_bytes(int R, int Hq, int Hkv, int D);
cudaError_t launch_attention(const moe_fp4_attention_args& a, cudaStream_t st);
cudaError_t attention_status_address(void** p);

}  // namespace moe_fp4
