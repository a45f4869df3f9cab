// The router's choice of experts (moe_fp4_route_topk): per token the top_k
// experts by logit (softmax) or by sigmoid(logit) + bias, ties to the lowest
// index, and their weights.  Experts with a logit of -inf or NaN are never
// chosen; a row that runs out of experts ends in id -1 with weight 0.
//
// A warp per token.  Up to 1024 experts the scores stay in registers as
// sortable integers, and a bound cuts them to a few candidates: the top_k-th
// largest of the lanes' own maxima is no larger than the top_k-th largest
// score, so only scores at or above it (about as many as top_k) are gathered
// in shared memory, and a candidate's place is the count of larger ones.
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

// The weights of the choices in lanes j < k (id -1: none) and their stores.
// `soft_total`: softmax only, the sum of exp(logit - top) over the row.
__device__ __forceinline__ void store_choice(const RouteArgs& a, int64_t m, int lane, int place, int id, float logit,
                                             float top, float soft_total) {
  const bool chosen = place < a.k && id >= 0;
  float w = 0.f;
  if (chosen) w = a.sigmoid ? sigmoid_exact(logit) : expf(logit - top);
  float total = a.sigmoid ? 1.f : soft_total;
  if (a.renormalize) {
    total = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (place < a.k) {
    a.ids[m * a.k + place] = chosen ? id : -1;
    a.weights[m * a.k + place] = !chosen || total == 0.f ? 0.f : __fdiv_rn(w, total) * a.scale;
  }
}

// A float's value from its order (order_key's inverse).
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}

constexpr int kRouteWarps = 8;

// At most 128 kGroups experts: lane l holds experts 128 g + 4 l + c.
template <int kGroups>
__global__ void __launch_bounds__(32 * kRouteWarps) route_topk_kernel(RouteArgs a, int vec) {
  __shared__ unsigned long long found[kRouteWarps][32];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t m = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (m >= a.M) return;
  // scores in order, 0 for experts that cannot be chosen
  uint32_t key[4 * kGroups];
  {
    float v[4 * kGroups];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int e = 128 * g + 4 * lane;
      if (vec && e + 4 <= a.E) {
        if (a.f32) {
          const float4 u = *reinterpret_cast<const float4*>(static_cast<const float*>(a.logits) + m * a.row + e);
          v[4 * g] = u.x, v[4 * g + 1] = u.y, v[4 * g + 2] = u.z, v[4 * g + 3] = u.w;
        } else {
          const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.logits) + m * a.row + e);
          v[4 * g] = __uint_as_float(u.x << 16), v[4 * g + 1] = __uint_as_float(u.x & 0xffff0000u);
          v[4 * g + 2] = __uint_as_float(u.y << 16), v[4 * g + 3] = __uint_as_float(u.y & 0xffff0000u);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) v[4 * g + c] = e + c < a.E ? route_logit(a, m, e + c) : -INFINITY;
      }
    }
#pragma unroll
    for (int i = 0; i < 4 * kGroups; ++i) {
      const int e = 128 * (i / 4) + 4 * lane + i % 4;
      key[i] = e < a.E ? (uint32_t)(route_key(a, v[i], e) >> 32) : 0u;
    }
  }
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < 4 * kGroups; ++i) mine = max(mine, key[i]);
  uint32_t bound = 0, best = 0;
  for (int j = 0; j < a.k; ++j) {
    bound = __reduce_max_sync(0xffffffffu, mine);
    if (j == 0) best = bound;
    if (bound == 0) break;
    if (mine == bound) mine = 0;
  }
  // (equal maxima leave together, which only lowers the bound)
  int n = 0;
  unsigned long long* list = found[threadIdx.x / 32];
#pragma unroll
  for (int i = 0; i < 4 * kGroups; ++i) {
    const bool in = key[i] >= bound && key[i] != 0;
    const uint32_t who = __ballot_sync(0xffffffffu, in);
    if (who == 0) continue;
    const int at = n + __popc(who & ((1u << lane) - 1u));
    if (in && at < 32)
      list[at] = ((unsigned long long)key[i] << 32) | (uint32_t)~(128 * (i / 4) + 4 * lane + i % 4);
    n += __popc(who);
  }
  __syncwarp();
  unsigned long long pick = 0;
  int place = 32;
  if (n <= 32) {
    // place = candidates above this lane's; lanes past the candidates take
    // the places after them
    pick = lane < n ? list[lane] : 0;
    place = lane < n ? 0 : lane;
    if (lane < n)
      for (int c = 0; c < n; ++c) place += list[c] > pick;
  } else {
    // many equal scores: one choice after another
    unsigned long long last = ~0ull;
    for (int j = 0; j < a.k; ++j) {
      unsigned long long top = 0;
#pragma unroll
      for (int i = 0; i < 4 * kGroups; ++i) {
        const unsigned long long full =
            ((unsigned long long)key[i] << 32) | (uint32_t)~(128 * (i / 4) + 4 * lane + i % 4);
        if (key[i] != 0 && full < last && full > top) top = full;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long other = __shfl_xor_sync(0xffffffffu, top, o);
        top = other > top ? other : top;
      }
      last = top;
      if (lane == j) pick = top, place = j;
    }
  }
  const int id = pick ? (int)~(uint32_t)pick : -1;
  // best: the largest score's order, with the softmax the largest logit's
  const float top = key_value(best);
  float total = 0.f;
  if (!a.sigmoid && !a.renormalize) {
#pragma unroll
    for (int i = 0; i < 4 * kGroups; ++i)
      if (key[i] != 0) total += expf(key_value(key[i]) - top);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  float logit = 0.f;
  if (id >= 0) logit = a.sigmoid ? route_logit(a, m, id) : key_value((uint32_t)(pick >> 32));
  store_choice(a, m, lane, place, id, logit, top, total);
}

// Any number of experts: each of the k choices is a pass over the row for the
// largest key below the last one.
__global__ void __launch_bounds__(32 * kRouteWarps) route_topk_wide_kernel(RouteArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t m = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (m >= a.M) return;
  unsigned long long last = ~0ull;
  int id = -1;  // lane j < k holds choice j
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
  const float top = __shfl_sync(0xffffffffu, logit, 0);  // (softmax: the first choice has the largest logit)
  float total = 0.f;
  if (!a.sigmoid && !a.renormalize) {
    for (int e = lane; e < a.E; e += 32) {
      const float v = route_logit(a, m, e);
      if (v > -INFINITY) total += expf(v - top);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  store_choice(a, m, lane, lane, id, logit, top, total);
}

cudaError_t launch_route_topk(const RouteArgs& a, cudaStream_t st) {
  int sms = 0;
  const cudaError_t e = current_device_sms(&sms);
  if (e != cudaSuccess) return e;
  const unsigned warps = a.M <= 4 * sms ? 2 : kRouteWarps;  // few tokens: spread over the SMs
  const unsigned grid = (unsigned)(((int64_t)a.M + warps - 1) / warps), threads = 32 * warps;
  const unsigned bytes = a.f32 ? 16 : 8;  // of a lane's four logits
  const int vec = ((uintptr_t)a.logits % bytes) == 0 && a.row % 4 == 0;
  if (a.E <= 128) return launch_dependent(route_topk_kernel<1>, grid, threads, st, a, vec);
  if (a.E <= 256) return launch_dependent(route_topk_kernel<2>, grid, threads, st, a, vec);
  if (a.E <= 512) return launch_dependent(route_topk_kernel<4>, grid, threads, st, a, vec);
  if (a.E <= 1024) return launch_dependent(route_topk_kernel<8>, grid, threads, st, a, vec);
  return launch_dependent(route_topk_wide_kernel, grid, threads, st, a);
}

}  // namespace moe_fp4
