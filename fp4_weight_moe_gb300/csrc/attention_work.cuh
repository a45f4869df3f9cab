// How an attention call's work is cut (attention.cu): shared by the kernels
// that attend and the one that joins their parts.
//
// A request's queries and the heads of one key head are its rows (query i,
// head g of the group: row i G + g), taken kRows at a time: a tile.  A tile
// and a key head are an item: its keys, from the first that any of its
// queries sees to the last, counted in units of kUnit tokens.  The units of
// all items lie in one line (by request, then tile, then key head), which the
// workers share evenly: each takes one stretch, so long rows are split over
// many workers and short ones fill one.  Only the first and the last item of
// a stretch can be shared with other workers; their sums go to the worker's
// two places in the workspace and are joined in the order of the workers.
#pragma once

#include "attention.cuh"

namespace moe_fp4 {

struct AttnArgs {
  moe_fp4_attention_args a;
  int group;      // Hq / Hkv
  int capacity;   // tokens that a table row holds
  float* parts;   // [2 workers][kRows][D] sums, then [2 workers][kRows][2] maximum and divisor
  int64_t* prefix;  // [R + 1] units before each request
  int workers;    // at most
  int least;      // units that are worth a worker
};

// A request of the batch.
struct AttnRequest {
  int row0, n, length;  // first row of q, queries, tokens in the cache
};

__device__ __forceinline__ AttnRequest attn_request(const AttnArgs& p, int r) {
  AttnRequest q;
  q.row0 = min(max(p.a.offsets[r], 0), p.a.T);
  q.n = max(min(p.a.offsets[r + 1], p.a.T) - q.row0, 0);
  q.length = max(p.a.lengths[r], 0);
  return q;
}

// The keys that rows [row, row + rows) of a request see: [lo, hi), in units.
struct AttnSpan {
  int lo, hi;        // tokens
  int first, units;  // unit of lo, number of units
};

template <int kUnit>
__device__ __forceinline__ AttnSpan attn_span(const AttnArgs& p, const AttnRequest& q, int row, int rows) {
  AttnSpan s;
  const int q0 = row / p.group, q1 = min((row + rows - 1) / p.group, q.n - 1);
  const int p0 = q.length - q.n + q0, p1 = q.length - q.n + q1;
  s.lo = p.a.window > 0 ? max(p0 - p.a.window + 1, 0) : 0;
  s.hi = min(p1 + 1, p.capacity);
  s.first = s.lo / kUnit;
  s.units = s.hi > s.lo ? (s.hi + kUnit - 1) / kUnit - s.first : 0;
  return s;
}

template <int kRows>
__device__ __forceinline__ int attn_tiles(const AttnArgs& p, const AttnRequest& q) {
  return (int)(((int64_t)q.n * p.group + kRows - 1) / kRows);
}

template <int kRows, int kUnit>
__device__ __forceinline__ int64_t attn_units(const AttnArgs& p, int r) {
  const AttnRequest q = attn_request(p, r);
  const int tiles = attn_tiles<kRows>(p, q);
  int64_t sum = 0;
  for (int i = 0; i < tiles; ++i) sum += attn_span<kUnit>(p, q, i * kRows, kRows).units;
  return sum * p.a.Hkv;
}

// Workers that share `units`, and the first unit of worker w.
__device__ __forceinline__ int attn_workers(const AttnArgs& p, int64_t units) {
  return (int)max(min((int64_t)p.workers, units / p.least), (int64_t)1);
}
__device__ __forceinline__ int64_t attn_start(int w, int64_t units, int workers) { return w * units / workers; }
// The worker that has unit u.
__device__ __forceinline__ int attn_owner(int64_t u, int64_t units, int workers) {
  return (int)(((u + 1) * workers - 1) / units);
}

// Sum over the block's threads of v before this thread's, and all of it.
template <int kThreads>
__device__ __forceinline__ int64_t block_before(int64_t v, int64_t* total, int64_t* shared) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t upto = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += x;
  }
  __syncthreads();
  if (lane == 31) shared[warp] = upto;
  __syncthreads();
  int64_t before = upto - v, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += shared[w];
    all += shared[w];
  }
  *total = all;
  return before;
}

}  // namespace moe_fp4
