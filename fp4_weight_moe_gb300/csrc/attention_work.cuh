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
#include "host.cuh"

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

// Many rows to a key head (attention_tc.cu), and its parts' room.
cudaError_t launch_attention_tc(const AttnArgs& p, int sms, cudaStream_t st);
size_t attention_tc_parts_bytes(int D, int sms);

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

// A place in the line: an item, and the unit of it.  The lanes of a warp keep
// one together.
template <int kRows, int kUnit>
struct AttnCursor {
  AttnRequest q;
  AttnSpan span;
  int r, tiles, tile, head, from;

  __device__ __forceinline__ void request(const AttnArgs& p, int request) {
    r = request;
    q = attn_request(p, r);
    tiles = attn_tiles<kRows>(p, q);
  }
  // `rest` units into request `request`, which has more than that
  __device__ __forceinline__ void start(const AttnArgs& p, int request_, int64_t rest) {
    request(p, request_);
    const int lane = threadIdx.x & 31;
    for (tile = 0;; tile += 32) {
      const int mine = tile + lane < tiles ? attn_span<kUnit>(p, q, (tile + lane) * kRows, kRows).units : 0;
      int64_t upto = (int64_t)mine * p.a.Hkv;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      const unsigned there = __ballot_sync(0xffffffffu, rest < upto);
      const int at = there ? __ffs(there) - 1 : 31;
      const int64_t before = __shfl_sync(0xffffffffu, upto - (int64_t)mine * p.a.Hkv, at);
      const int64_t all = __shfl_sync(0xffffffffu, upto, 31);
      if (there) {
        tile += at;
        rest -= before;
        break;
      }
      rest -= all;
      if (tile + 32 >= tiles) break;  // (not reached)
    }
    span = attn_span<kUnit>(p, q, tile * kRows, kRows);
    head = (int)(rest / max(span.units, 1));
    from = (int)(rest - (int64_t)head * span.units);
  }
  // the next item of the line, of which there is one
  __device__ __forceinline__ void next(const AttnArgs& p) {
    from = 0;
    if (++head < p.a.Hkv) return;
    head = 0;
    do {
      if (++tile >= tiles) {
        if (r + 1 >= p.a.R) return;  // (not reached)
        request(p, r + 1);
        tile = 0;
        if (tiles == 0) span.units = 0;
      }
      if (tile < tiles) span = attn_span<kUnit>(p, q, tile * kRows, kRows);
    } while (span.units == 0);
  }
  __device__ __forceinline__ int rows(const AttnArgs& p) const {
    return (int)min((int64_t)kRows, (int64_t)q.n * p.group - (int64_t)tile * kRows);
  }
};

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

// Every CTA finds the line's length and its worker's stretch [u, u_end) of it
// (CTA 0 writes down the sums before each request); false where it has none.
template <int kRows, int kUnit, int kThreads>
__device__ __forceinline__ bool attn_stretch(const AttnArgs& p, AttnCursor<kRows, kUnit>& cursor, int64_t& u,
                                             int64_t& u_end) {
  __shared__ int64_t shared[kThreads / 32];
  __shared__ int64_t found_rest;
  __shared__ int found;
  const int each = ceil_div(max(p.a.R, 1), kThreads);
  const int r0 = min((int)threadIdx.x * each, p.a.R), r1 = min(r0 + each, p.a.R);
  int64_t mine = 0, units;
  for (int r = r0; r < r1; ++r) mine += attn_units<kRows, kUnit>(p, r);
  const int64_t before = block_before<kThreads>(mine, &units, shared);
  if (blockIdx.x == 0) {
    int64_t at = before;
    for (int r = r0; r < r1; ++r) {
      p.prefix[r] = at;
      if (r + 1 < r1) at += attn_units<kRows, kUnit>(p, r);
    }
    if (threadIdx.x == 0) p.prefix[p.a.R] = units;
  }
  const int workers = attn_workers(p, units);
  if (units == 0 || (int)blockIdx.x >= workers) return false;
  u = attn_start(blockIdx.x, units, workers);
  u_end = attn_start(blockIdx.x + 1, units, workers);
  if (before <= u && u < before + mine) {
    int64_t at = before;
    int r = r0;
    for (; r + 1 < r1; ++r) {
      const int64_t n = attn_units<kRows, kUnit>(p, r);
      if (u < at + n) break;
      at += n;
    }
    found = r;
    found_rest = u - at;
  }
  __syncthreads();
  cursor.start(p, found, found_rest);
  return true;
}

// ---------------------------------------------------------------- pieces of the kernels
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The power of two that brings a row's largest |q| to [2^14, 2^15), and its inverse.
__device__ __forceinline__ float row_scale(float top, float& back) {
  const int e = min(max((int)((__float_as_uint(top) >> 23) & 0xff) - 127 - 14, -100), 100);
  back = __uint_as_float((uint32_t)(127 + e) << 23);
  return __uint_as_float((uint32_t)(127 - e) << 23);
}

// A row's last step: from its maximum (units of log 2) and divisor, with the
// sink's term, the factor of its sums, and its lse.
__device__ __forceinline__ float attn_finish(const AttnArgs& p, int head, float top, float sum, float& lse) {
  float by = 1.f;
  if (p.a.sinks) {
    const float sink = p.a.sinks[head] * kLog2e, next = fmaxf(top, sink);
    if (next != -INFINITY) {
      // (a maximum of -inf: no key, or none but NaN scores)
      by = top == -INFINITY ? (sum == sum ? 0.f : 1.f) : exp2_approx(top - next);
      sum = sum * by + exp2_approx(sink - next);
      top = next;
    }
  }
  lse = sum == 0.f ? -INFINITY : (top == -INFINITY ? 0.f : top) * kLn2 + logf(sum);
  return sum == 0.f ? 0.f : p.a.v_scale * by / sum;
}

__device__ __forceinline__ __nv_bfloat16* attn_out(const AttnArgs& p, int token, int head) {
  return static_cast<__nv_bfloat16*>(p.a.out) + (int64_t)token * p.a.out_row + (int64_t)head * p.a.out_head;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// Where a part's maximum and divisor lie, behind the sums.
template <int D, int kRows>
__device__ __forceinline__ float* attn_stats(const AttnArgs& p, int64_t part, int row) {
  return p.parts + (int64_t)2 * p.workers * kRows * D + (part * kRows + row) * 2;
}

// CTAs x < workers: x joins the parts of the item that its stretch begins in
// the middle of, if no earlier stretch does, in the workers' order, kJoinRows
// rows of it.  The others write the rows that no worker has: queries that see
// no key, and rows behind the last sequence.
constexpr int kJoinRows = 32, kJoinThreads = 256;

template <int D, int kRows, int kUnit>
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(AttnArgs p) {
  pdl_wait();
  pdl_launch_dependents();
  if ((int)blockIdx.x < p.workers) {
    const int64_t units = p.prefix[p.a.R];
    const int workers = attn_workers(p, units), w = blockIdx.x;
    if (w == 0 || w >= workers || units == 0) return;
    const int64_t u = attn_start(w, units, workers);
    int lo = 0, hi = p.a.R;  // prefix[lo] <= u < prefix[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.prefix[mid] <= u)
        lo = mid;
      else
        hi = mid;
    }
    AttnCursor<kRows, kUnit> c;
    c.start(p, lo, u - p.prefix[lo]);
    const int64_t u0 = u - c.from;
    if (c.from == 0 || attn_start(w - 1, units, workers) > u0) return;
    const int last = attn_owner(u0 + c.span.units - 1, units, workers);
    const int row0 = blockIdx.y * kJoinRows, rows = min(c.rows(p) - row0, kJoinRows);
    for (int i = threadIdx.x; i < rows * (D / 4); i += kJoinThreads) {
      const int row = row0 + i / (D / 4), d = 4 * (i % (D / 4));
      float top = -INFINITY, sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int x = w - 1; x <= last; ++x) {
        const int64_t part = 2 * (int64_t)x + (x == w - 1 ? 1 : 0);
        const float2 st = *reinterpret_cast<const float2*>(attn_stats<D, kRows>(p, part, row));
        const float4 v = *reinterpret_cast<const float4*>(p.parts + (part * kRows + row) * D + d);
        const float next = fmaxf(top, st.x);
        const float old_by = top == next ? 1.f : exp2_approx(top - next);
        const float new_by = st.x == next ? 1.f : exp2_approx(st.x - next);
        top = next;
        sum = sum * old_by + st.y * new_by;
        acc.x = acc.x * old_by + v.x * new_by;
        acc.y = acc.y * old_by + v.y * new_by;
        acc.z = acc.z * old_by + v.z * new_by;
        acc.w = acc.w * old_by + v.w * new_by;
      }
      const int rr = c.tile * kRows + row, token = c.q.row0 + rr / p.group, hq = c.head * p.group + rr % p.group;
      float lse;
      const float inv = attn_finish(p, hq, top, sum, lse);
      *reinterpret_cast<uint2*>(attn_out(p, token, hq) + d) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (p.a.lse && d == 0) p.a.lse[(int64_t)token * p.a.Hq + hq] = lse;
    }
    return;
  }
  if (blockIdx.y > 0) return;
  const int token = (blockIdx.x - p.workers) * kJoinThreads + threadIdx.x;
  bool none = false, inside = false;  // sees no key; is a request's
  if (token < p.a.T) {
    inside = p.a.R > 0 && token >= p.a.offsets[0] && token < p.a.offsets[p.a.R];
    none = !inside;
    if (inside) {
      int lo = 0, hi = p.a.R;  // offsets[lo] <= token < offsets[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.a.offsets[mid] <= token)
          lo = mid;
        else
          hi = mid;
      }
      const AttnRequest q = attn_request(p, lo);
      none = attn_span<1>(p, q, (token - q.row0) * p.group, p.group).units == 0;
    }
  }
  const int warp0 = token - (threadIdx.x & 31), lane = threadIdx.x & 31;
  const unsigned real = __ballot_sync(0xffffffffu, inside);
  for (unsigned todo = __ballot_sync(0xffffffffu, none); todo; todo &= todo - 1) {
    const int at = __ffs(todo) - 1, t = warp0 + at;
    for (int i = lane; i < p.a.Hq * (D / 8); i += 32)
      *reinterpret_cast<uint4*>(attn_out(p, t, i / (D / 8)) + 8 * (i % (D / 8))) = make_uint4(0, 0, 0, 0);
    if (p.a.lse)
      for (int h = lane; h < p.a.Hq; h += 32)
        p.a.lse[(int64_t)t * p.a.Hq + h] = (real >> at & 1u) && p.a.sinks ? p.a.sinks[h] : -INFINITY;
  }
}

template <int D, int kRows, int kUnit>
cudaError_t launch_attention_join(const AttnArgs& p, cudaStream_t st) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(p.workers + ceil_div(p.a.T, kJoinThreads)), (unsigned)ceil_div(kRows, kJoinRows));
  c.blockDim = dim3(kJoinThreads);
  c.stream = st;
  c.attrs = at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, attention_join_kernel<D, kRows, kUnit>, p);
}

}  // namespace moe_fp4
