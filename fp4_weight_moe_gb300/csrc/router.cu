// The router's choice of experts (moe_fp4_route_topk): per token the top_k
// experts by logit (softmax) or by sigmoid(logit) + bias, ties to the lowest
// index, and their weights.  Experts with a logit of -inf or NaN are never
// chosen; a row that runs out of experts ends in id -1 with weight 0.  With
// the softmax +inf comes first, and its row's weights are NaN (inf - inf).
//
// A warp per token.  A bound cuts the scores, as sortable integers, to a few
// candidates: the top_k-th largest of the lanes' two best each is no larger
// than the top_k-th largest score, so only scores at or above it (hardly more
// than top_k) are gathered in shared memory, and a candidate's place is the
// count of larger ones.  Up to 1024 experts the scores stay in registers; past that
// a second pass over the row finds the candidates.
//
// The two best, not the best alone: with one a lane, top_k = 16 of 32 lanes
// left more than the list's 32 candidates in one row of a hundred or so, and
// those rows' 16 passes set the time (M = 1024, 512 experts: 5.7 us, now 3.1;
// top_k = 10, where the list held: 4.9 us at M = 4096, now 5.1).
//
// Bound: few tokens, the chain of one row (2.4 us at M = 4, 3.5 with 288
// sigmoids, from a graph), and so up to a wave of CTAs (M = 4096, 512 experts:
// 512 CTAs for 608 places, 5.1 us, sigmoid 7.5; issue slots 30 and 39 % busy
// over the whole launch); many, the instructions of the scores (M = 32768, 512
// experts in FP32: 27 us of which the logits' bytes are 10; sigmoid 42; issue
// slots 81 and 83 % busy while SMs are).  An IEEE reciprocal for every sigmoid,
// a branch each, took 4.8 us at M = 4, E = 288 where recip_rn takes 3.5.
#include "block.cuh"
#include "fp8_quant.cuh"
#include "host.cuh"

namespace moe_fp4 {

// A float's order as an unsigned integer; -0 and +0 alike.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// 1 / (1 + e^-v), each step rounded (the reciprocal correctly: the quotient).
__device__ __forceinline__ float sigmoid_exact(float v) { return __frcp_rn(1.0f + expf(-v)); }

__device__ __forceinline__ float route_logit(const RouteArgs& a, int64_t m, int e) {
  return a.f32 ? static_cast<const float*>(a.logits)[m * a.row + e]
               : __uint_as_float((uint32_t) static_cast<const uint16_t*>(a.logits)[m * a.row + e] << 16);
}

// The order of an expert's score, 0 if it cannot be chosen.
__device__ __forceinline__ uint32_t score_key(float logit, float score) {
  return logit > -INFINITY && score == score ? order_key(score) : 0u;
}

// The sort key of expert e, 0 if it cannot be chosen: the score's order above
// the complement of the index, so that the largest key is the best score and
// among equals the lowest index.
__device__ __forceinline__ unsigned long long route_key(const RouteArgs& a, float logit, int e) {
  float v = logit;
  if (a.sigmoid) {
    const float x = 1.0f + expf(-logit);
    v = x < 0x1p126f ? recip_rn(x) : __frcp_rn(x);
    if (a.bias) v += a.bias[e];
  }
  const uint32_t k = score_key(logit, v);
  return k ? ((unsigned long long)k << 32) | (uint32_t)~e : 0;
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

// The two best of a lane's scores.
struct LaneBest {
  uint32_t first = 0, second = 0;
  __device__ __forceinline__ void add(uint32_t key) {
    second = max(second, min(first, key));
    first = max(first, key);
  }
};

// The k-th largest of the lanes' two best (0: there are fewer; equal ones of
// several lanes leave together, which only lowers the bound).  *best: the
// largest.
__device__ __forceinline__ uint32_t candidate_bound(LaneBest mine, int k, uint32_t* best) {
  uint32_t bound = 0;
  for (int j = 0; j < k; ++j) {
    bound = __reduce_max_sync(0xffffffffu, mine.first);
    if (j == 0) *best = bound;
    if (bound == 0) break;
    if (mine.first == bound) mine.first = mine.second, mine.second = 0;
  }
  return bound;
}

// This lane's candidate of n <= 32 (0: none) and its place: the count of
// larger ones; lanes past the candidates take the places after them.
__device__ __forceinline__ unsigned long long candidate_place(const unsigned long long* list, int n, int lane,
                                                              int* place) {
  const unsigned long long pick = lane < n ? list[lane] : 0;
  *place = lane < n ? 0 : lane;
  if (lane < n) {
#pragma unroll 4
    for (int c = 0; c < n; ++c) *place += list[c] > pick;
  }
  return pick;
}

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
    if (a.sigmoid) {
      float score[4 * kGroups];
      bool fast = true;
#pragma unroll
      for (int i = 0; i < 4 * kGroups; ++i) {
        const float x = 1.0f + expf(-v[i]);
        fast = fast && (x < 0x1p126f || !(v[i] > -INFINITY));  // (what cannot be chosen may come out as anything)
        score[i] = recip_rn(x);
      }
      if (!__all_sync(0xffffffffu, fast)) {
#pragma unroll
        for (int i = 0; i < 4 * kGroups; ++i) score[i] = sigmoid_exact(v[i]);
      }
      if (a.bias) {
#pragma unroll
        for (int i = 0; i < 4 * kGroups; ++i) {
          const int e = 128 * (i / 4) + 4 * lane + i % 4;
          if (e < a.E) score[i] += a.bias[e];
        }
      }
#pragma unroll
      for (int i = 0; i < 4 * kGroups; ++i) key[i] = score_key(v[i], score[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4 * kGroups; ++i) key[i] = score_key(v[i], v[i]);
    }
  }
  LaneBest mine;
#pragma unroll
  for (int i = 0; i < 4 * kGroups; ++i) mine.add(key[i]);
  uint32_t best = 0;
  const uint32_t bound = candidate_bound(mine, a.k, &best);
  // gathered lane by lane: each lane's place is the count in the lanes before
  unsigned long long* list = found[threadIdx.x / 32];
  int n = 0;
#pragma unroll
  for (int i = 0; i < 4 * kGroups; ++i) n += key[i] >= bound && key[i] != 0;
  int at = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int before = __shfl_up_sync(0xffffffffu, at, o);
    if (lane >= o) at += before;
  }
  const int end = at;
  at -= n;
  n = __shfl_sync(0xffffffffu, end, 31);
  if (n <= 32) {
#pragma unroll
    for (int i = 0; i < 4 * kGroups; ++i)
      if (key[i] >= bound && key[i] != 0)
        list[at++] = ((unsigned long long)key[i] << 32) | (uint32_t)~(128 * (i / 4) + 4 * lane + i % 4);
  }
  __syncwarp();
  unsigned long long pick = 0;
  int place = 32;
  if (n <= 32) {
    pick = candidate_place(list, n, lane, &place);
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

// Any number of experts: a pass for the lanes' best and one for the
// candidates (M = 64, 4096 experts, top_k 8: 26 us, sigmoid 64: a warp's own
// chain of loads and scores).
__global__ void __launch_bounds__(32 * kRouteWarps) route_topk_wide_kernel(RouteArgs a) {
  __shared__ unsigned long long found[kRouteWarps][32];
  pdl_wait();
  pdl_launch_dependents();
  const int64_t m = (int64_t)blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x & 31;
  if (m >= a.M) return;
  LaneBest mine;
#pragma unroll 8
  for (int e = lane; e < a.E; e += 32) mine.add((uint32_t)(route_key(a, route_logit(a, m, e), e) >> 32));
  uint32_t best = 0;
  const uint32_t bound = candidate_bound(mine, a.k, &best);
  unsigned long long* list = found[threadIdx.x / 32];
  int n = 0;
#pragma unroll 4
  for (int e0 = 0; e0 < a.E; e0 += 32) {
    const int e = e0 + lane;
    const unsigned long long key = e < a.E ? route_key(a, route_logit(a, m, e), e) : 0;
    const bool in = key != 0 && (uint32_t)(key >> 32) >= bound;
    const uint32_t votes = __ballot_sync(0xffffffffu, in);
    const int at = n + __popc(votes & ((1u << lane) - 1));
    if (in && at < 32) list[at] = key;
    n += __popc(votes);
  }
  __syncwarp();
  unsigned long long pick = 0;
  int place = 32;
  if (n <= 32) {
    pick = candidate_place(list, n, lane, &place);
  } else {
    // many equal scores: each choice is a pass for the largest key below the last
    unsigned long long last = ~0ull;
    place = lane;
    for (int j = 0; j < a.k; ++j) {
      unsigned long long top = 0;
      for (int e = lane; e < a.E; e += 32) {
        const unsigned long long key = route_key(a, route_logit(a, m, e), e);
        if (key < last && key > top) top = key;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long other = __shfl_xor_sync(0xffffffffu, top, o);
        top = other > top ? other : top;
      }
      if (top == 0) break;
      last = top;
      if (lane == j) pick = top;
    }
  }
  const int id = pick ? (int)~(uint32_t)pick : -1;
  const float logit = id >= 0 ? route_logit(a, m, id) : 0.f;
  const float top = key_value(best);  // (softmax: the largest logit)
  float total = 0.f;
  if (!a.sigmoid && !a.renormalize) {
    for (int e = lane; e < a.E; e += 32) {
      const float v = route_logit(a, m, e);
      if (v > -INFINITY) total += expf(v - top);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  store_choice(a, m, lane, place, id, logit, top, total);
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
