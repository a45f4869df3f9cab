// The paged cache's step (block tables, slots and positions from request
// lengths: moe_fp4_cache_step) and its reader (moe_fp4_cache_read).
//
// The step is three running sums over the requests (new tokens, pages given
// back, pages asked for), then pages moved between the table and the stack of
// free ones, then a place for each token.  The first launch is one CTA: the
// pages that it takes may be those that it has just put on the stack.  A few
// tokens it places itself; many are placed by a second launch, whose threads
// each find their request by bisection.
//
// Bound by latency, a handful of dependent reads: 64 requests of a token each
// 3.5 us, 512 requests of 65536 new tokens 9.1.  Requests lie next to one
// another in a warp, which moves the pages of one after the other's: few
// requests with many pages are slow (pages of 16 tokens: 32 prompts of 2048
// tokens 29 us; 2 requests of 262144 tokens that end 196, 32 of them 3.1 ms).
// The reader moves 0.56 + 2 bytes a value: 8192 tokens of 8 heads of 128
// columns, keys and values, 11 us between other calls of its own, behind the
// store 13; its two halves are loaded one after the other.
#include "attention.cuh"
#include "host.cuh"

namespace moe_fp4 {
namespace {

constexpr int kStepThreads = 1024;
// Pages that a lane takes for its request by itself (512 requests of two pages
// each, a warp to one after the other: 14 us of the step's 15).
constexpr int kFew = 4;
// Tokens that the one CTA places itself (64 tokens 3.4 us, with a second launch
// 4.8; 512 requests of up to 2 tokens 6.4 and 7.8, of up to 8 9.4 and 8.4).
constexpr int kStepTokens = 2 * kStepThreads;

struct Sums {
  int fresh, back, need;
};

__device__ __forceinline__ Sums operator+(Sums a, Sums b) { return {a.fresh + b.fresh, a.back + b.back, a.need + b.need}; }

__device__ __forceinline__ Sums shuffle_up(Sums v, int o) {
  return {__shfl_up_sync(0xffffffffu, v.fresh, o), __shfl_up_sync(0xffffffffu, v.back, o),
          __shfl_up_sync(0xffffffffu, v.need, o)};
}

// A request before the step: its tokens, pages, and what it asks for.
struct Request {
  int length, fresh, have, need;  // length and pages after its release; need -1: more than its table row holds
  int back;                       // pages that it gives back
};

__device__ __forceinline__ Request request(const moe_fp4_cache_step_args& a, int r) {
  Request q;
  const int p = a.page_size;
  q.length = max(a.lengths[r], 0);
  q.fresh = max(a.new_tokens[r], 0);
  q.back = 0;
  if (a.finished && a.finished[r]) {
    q.back = (int)min(((int64_t)q.length + p - 1) / p, (int64_t)a.table_width);
    q.length = 0;
  }
  q.have = (int)(((int64_t)q.length + p - 1) / p);
  const int64_t pages = ((int64_t)q.length + q.fresh + p - 1) / p;
  q.need = pages > a.table_width && q.fresh > 0 ? -1 : (int)(pages - q.have);
  return q;
}

// Where token t < offsets[R] goes.
__device__ __forceinline__ void place(const moe_fp4_cache_step_args& a, const int32_t* offsets, int t) {
  if (t >= offsets[a.R]) {
    a.positions[t] = 0;
    a.slots[t] = -1;
    return;
  }
  int lo = 0, hi = a.R;  // offsets[lo] <= t < offsets[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int taken = a.accepted[lo];
  const int pos = a.lengths_out[lo] - taken + (t - offsets[lo]);
  a.positions[t] = pos;
  a.slots[t] = taken > 0 ? (int64_t)a.tables[lo * a.table_row + pos / a.page_size] * a.page_size + pos % a.page_size
                         : -1;
}

__global__ void __launch_bounds__(kStepThreads) cache_step_kernel(moe_fp4_cache_step_args a, bool places) {
  __shared__ Sums warp_sums[kStepThreads / 32];
  __shared__ int top_out;
  pdl_wait();
  pdl_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int each = ceil_div(max(a.R, 1), kStepThreads);
  const int r0 = min(tid * each, a.R), r1 = min(r0 + each, a.R);

  Sums mine = {0, 0, 0};
  for (int r = r0; r < r1; ++r) {
    const Request q = request(a, r);
    mine = mine + Sums{q.fresh, q.back, max(q.need, 0)};
  }
  Sums upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Sums v = shuffle_up(upto, o);
    if (lane >= o) upto = upto + v;
  }
  if (lane == 31) warp_sums[warp] = upto;
  if (tid == 0) top_out = 0;
  __syncthreads();
  if (warp == 0) {
    Sums w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Sums v = shuffle_up(w, o);
      if (lane >= o) w = w + v;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  Sums before = {upto.fresh - mine.fresh, upto.back - mine.back, upto.need - mine.need};
  if (warp > 0) before = before + warp_sums[warp - 1];
  const int count = max(min(*a.free_count, a.free_capacity), 0);
  const int top = min(count + warp_sums[kStepThreads / 32 - 1].back, a.free_capacity);

  // Pages given back: rows of the warp's lanes in turn, each by the whole warp.
  Sums at = before;
  for (int i = 0; i < each; ++i) {
    const int r = r0 + i;
    const int n = r < r1 ? request(a, r).back : 0;
    for (unsigned todo = __ballot_sync(0xffffffffu, n > 0); todo; todo &= todo - 1) {
      const int from = __ffs(todo) - 1;
      const int row = __shfl_sync(0xffffffffu, r, from), m = __shfl_sync(0xffffffffu, n, from);
      const int to = count + __shfl_sync(0xffffffffu, at.back, from);
      for (int j = lane; j < m; j += 32)
        if (to + j < a.free_capacity) a.free_pages[to + j] = a.tables[row * a.table_row + j];
    }
    at.back += n;
  }
  __syncthreads();

  // Pages taken, from the stack's top.
  for (int i = 0; i < each; ++i) {
    const int r = r0 + i;
    int n = 0, have = 0, need = 0;
    if (r < r1) {
      const Request q = request(a, r);
      need = max(q.need, 0);
      const bool takes = q.need == 0 || (q.need > 0 && at.need + need <= top);
      n = takes ? need : 0;
      have = q.have;
      a.offsets[r] = at.fresh;
      a.accepted[r] = takes ? q.fresh : 0;
      a.lengths_out[r] = q.length + (takes ? q.fresh : 0);
      at.fresh += q.fresh;
      if (n > 0) atomicMax(&top_out, at.need + n);  // (what was taken: accepted demands form a prefix of the sums)
    }
    // a lane takes its request's first few; a whole warp what is left
    int32_t pages[kFew];
#pragma unroll
    for (int j = 0; j < kFew; ++j)
      if (j < n) pages[j] = a.free_pages[top - 1 - at.need - j];
#pragma unroll
    for (int j = 0; j < kFew; ++j)
      if (j < n) a.tables[r * a.table_row + have + j] = pages[j];
    for (unsigned todo = __ballot_sync(0xffffffffu, n > kFew); todo; todo &= todo - 1) {
      const int from = __ffs(todo) - 1;
      const int row = __shfl_sync(0xffffffffu, r, from), m = __shfl_sync(0xffffffffu, n, from);
      const int first = __shfl_sync(0xffffffffu, have, from);
      const int next = top - 1 - __shfl_sync(0xffffffffu, at.need, from);
      for (int j = kFew + lane; j < m; j += 32) a.tables[row * a.table_row + first + j] = a.free_pages[next - j];
    }
    at.need += need;
  }
  if (tid == 0) a.offsets[a.R] = warp_sums[kStepThreads / 32 - 1].fresh;
  __syncthreads();
  if (tid == 0) *a.free_count_out = top - top_out;
  if (places)
    for (int t = tid; t < a.tokens; t += kStepThreads) place(a, a.offsets, t);
}

__global__ void __launch_bounds__(256) cache_place_kernel(moe_fp4_cache_step_args a) {
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.x * 256 + threadIdx.x;
  if (t < a.tokens) place(a, a.offsets, t);
}

// A token's head on D / 8 lanes, eight columns each.
template <int D>
__global__ void __launch_bounds__(256) cache_read_kernel(const uint8_t* cache, int64_t slots_max, int page_size,
                                                         int Hkv, const int64_t* slots, float k_scale, float v_scale,
                                                         uint4* k_out, uint4* v_out, int T) {
  constexpr int kLanes = D / 8;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t unit = i / kLanes;
  const int l = (int)(i % kLanes);
  if (unit >= (int64_t)T * Hkv) return;
  const int64_t slot = slots[unit / Hkv];
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    uint32_t w[4] = {0, 0, 0, 0};
    if (slot >= 0 && slot < slots_max) {
      const CachePlace p = cache_place(slot, (int)(unit % Hkv), Hkv, page_size, D);
      const uint8_t* half = cache + kind * cache_half_bytes(D);
      const uint32_t codes = *reinterpret_cast<const uint32_t*>(half + p.codes + 4 * l);
      const float s = e4m3_to_float(half[p.scales + l / 2]), by = kind ? v_scale : k_scale;
      uint32_t h[4];
      e2m1x8_to_half2x4(codes, h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 v = half2_bits_to_float2(h[j]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(v.x * s * by, v.y * s * by);
        w[j] = *reinterpret_cast<const uint32_t*>(&b);
      }
    }
    (kind ? v_out : k_out)[i] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

}  // namespace

cudaError_t launch_cache_step(const moe_fp4_cache_step_args& a, cudaStream_t st) {
  const bool places = a.tokens <= kStepTokens;
  const cudaError_t e = launch_dependent(cache_step_kernel, 1, kStepThreads, st, a, places);
  if (e != cudaSuccess || places) return e;
  return launch_dependent(cache_place_kernel, (unsigned)ceil_div(a.tokens, 256), 256, st, a);
}

template <int D>
static cudaError_t read_dim(const uint8_t* cache, int64_t slots_max, int page_size, int Hkv, const int64_t* slots,
                            float k_scale, float v_scale, void* k_out, void* v_out, int T, cudaStream_t st) {
  const int64_t grid = ((int64_t)T * Hkv * (D / 8) + 255) / 256;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_dependent(cache_read_kernel<D>, (unsigned)grid, 256, st, cache, slots_max, page_size, Hkv, slots,
                          k_scale, v_scale, static_cast<uint4*>(k_out), static_cast<uint4*>(v_out), T);
}

cudaError_t launch_cache_read(const uint8_t* cache, int64_t slots_max, int page_size, int Hkv, int D,
                              const int64_t* slots, float k_scale, float v_scale, void* k_out, void* v_out, int T,
                              cudaStream_t st) {
  switch (D) {
    case 64: return read_dim<64>(cache, slots_max, page_size, Hkv, slots, k_scale, v_scale, k_out, v_out, T, st);
    case 128: return read_dim<128>(cache, slots_max, page_size, Hkv, slots, k_scale, v_scale, k_out, v_out, T, st);
    default: return read_dim<256>(cache, slots_max, page_size, Hkv, slots, k_scale, v_scale, k_out, v_out, T, st);
  }
}

}  // namespace moe_fp4
