// The router's choice of experts (moe_fp4_route_topk): per token the top_k
// experts by logit (softmax) or by sigmoid(logit) + bias, ties to the lowest
// index, and their weights.  Experts with a logit of -inf or NaN are never
// chosen; a row that runs out of experts ends in id -1 with weight 0.
#include "block.cuh"
#include "host.cuh"

namespace moe_fp4 {

// A float's order as an unsigned integer; -0 and +0 alike.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float sigmoid_exact(float v) { return __fdiv_rn(1.0f, 1.0f + expf(-v)); }

__device__ __forceinline__ float route_logit(const RouteArgs& a, int64_t m, int e) {
  return a.f32 ? static_cast<const float*>(a.logits)[m * a.row + e]
               : __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.logits)[m * a.row + e] << 16);
}

// The sort key of expert e, 0 if it cannot be chosen: the score's order above
// the complement of the index, so that the largest key is the best score and
// among equals the lowest index.
__device__ __forceinline__ unsigned long long route_key(const RouteArgs& a, float logit, int e) {
  if (!(logit > -INFINITY)) return 0;
  float v = logit;
  if (a.sigmoid) {
    v = sigmoid_exact(logit);
    if (a.bias) v += a.bias[e];
    if (!(v == v)) return 0;
  }
  return ((unsigned long long)order_key(v) << 32) | (uint32_t)~e;
}

// A warp per token; each of the k choices is a pass over the row for the
// largest key below the last one.
__global__ void __launch_bounds__(256) route_topk_kernel(RouteArgs a) {
  const int64_t m = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) / 32;
  const int lane = threadIdx.x & 31;
  if (m >= a.M) return;
  unsigned long long last = ~0ull;
  int id = -1;        // lane j < k holds choice j
  float logit = 0.f;
  for (int j = 0; j < a.k; ++j) {
    unsigned long long best = 0;
    for (int e = lane; e < a.E; e += 32) {
      const unsigned long long key = route_key(a, route_logit(a, m, e), e);
      if (key < last && key > best) best = key;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const unsigned long long other = __shfl_xor_sync(0xffffffffu, best, o);
      best = other > best ? other : best;
    }
    if (best == 0) break;
    last = best;
    if (lane == j) {
      id = (int)~(uint32_t)best;
      logit = route_logit(a, m, id);
    }
  }
  float w = 0.f, total = 0.f;
  if (a.sigmoid) {
    if (id >= 0) w = sigmoid_exact(logit);
  } else {
    float top = -INFINITY;
    if (a.renormalize) {
      top = __shfl_sync(0xffffffffu, logit, 0);
    } else {
      for (int e = lane; e < a.E; e += 32) top = fmaxf(top, route_logit(a, m, e));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      for (int e = lane; e < a.E; e += 32) {
        const float v = route_logit(a, m, e);
        if (v > -INFINITY) total += expf(v - top);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if (id >= 0) w = expf(logit - top);
  }
  if (a.renormalize) {
    total = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  } else if (a.sigmoid) {
    total = 1.f;
  }
  if (lane < a.k) {
    a.ids[m * a.k + lane] = id;
    a.weights[m * a.k + lane] = id < 0 || total == 0.f ? 0.f : __fdiv_rn(w, total) * a.scale;
  }
}

cudaError_t launch_route_topk(const RouteArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)(((int64_t)a.M + 7) / 8);
  route_topk_kernel<<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace moe_fp4
