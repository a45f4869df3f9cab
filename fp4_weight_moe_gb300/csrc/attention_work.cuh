// How an attention call's work is cut (attention.cu, attention_tc.cu): shared
// by the kernels that attend and the one that joins their parts.
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
//
// A worker is a CTA, or each of its warps (kTeams, where the items are short:
// a CTA's warps would wait for each other at every item).  Items of at most
// kWhole units are not shared: they are their first unit's worker's.
#pragma once

#include "attention.cuh"
#include "host.cuh"

namespace moe_fp4 {

// What the workers leave for the join.
struct AttnLine {
  int64_t units, each;  // stretches are whole grains: `each`, and one more for the first `more` workers
  int more, workers, grain_log;
};
struct AttnPlace {  // where a worker's stretch begins
  int row0, first, tile, head, rows, from, units;  // first: position of the request's first query
};

struct AttnArgs {
  moe_fp4_attention_args a;
  int group, inverse; // Hq / Hkv, and 2^16 over it, rounded up
  int capacity;      // tokens that a table row holds
  float* parts;      // [2 workers][kRows][D] sums, then [2 workers][kRows][2] maximum and divisor
  AttnLine* line;
  AttnPlace* places; // [workers]
  int workers;       // at most
  int least;         // units that are worth a worker (an item always is)
};

// Many rows to a key head (attention_tc.cu; `rows`: of an average request), and
// its parts' room.
cudaError_t launch_attention_tc(const AttnArgs& p, int rows, int sms, cudaStream_t st);
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

// Rows of a tile as queries and heads of the group.
struct AttnRows {
  int query, head;  // of the tile's first row
};
__device__ __forceinline__ AttnRows attn_rows(const AttnArgs& p, int row) {
  const int query = row / p.group;
  return {query, row - query * p.group};
}
// Row `row` of the tile (a division of less than 1024 by at most 64: exact).
__device__ __forceinline__ AttnRows attn_row(const AttnArgs& p, const AttnRows& first, int row) {
  const int at = first.head + row, query = (at * p.inverse) >> 16;
  return {first.query + query, at - query * p.group};
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
  s.lo = p.a.window > 0 ? max(max(p0, 0) - p.a.window + 1, 0) : 0;  // (p0 -n at least: its difference stays in 32 bits)
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

__device__ __forceinline__ int64_t attn_quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;  // (both are not negative)
}

// A place in the line: an item, and the unit of it.  The lanes of a warp keep
// one together.
template <int kRows, int kUnit_, int kWhole_>
struct AttnCursor {
  static constexpr int kUnit = kUnit_, kWhole = kWhole_;
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
    head = (int)attn_quotient(rest, max(span.units, 1));
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

__device__ __forceinline__ AttnLine attn_line(int64_t units, int workers, int grain_log) {
  const int64_t grains = (units + (1 << grain_log) - 1) >> grain_log;
  AttnLine line = {units, attn_quotient(grains, workers), 0, workers, grain_log};
  line.more = (int)(grains - line.each * workers);
  return line;
}
// The first unit of worker w.
__device__ __forceinline__ int64_t attn_start(const AttnLine& line, int w) {
  return min((w * line.each + min(w, line.more)) << line.grain_log, line.units);
}
// The worker that has unit u.
__device__ __forceinline__ int attn_owner(const AttnLine& line, int64_t u) {
  const int64_t grain = u >> line.grain_log, longer = (line.each + 1) * line.more;
  return grain < longer ? (int)attn_quotient(grain, line.each + 1)
                        : line.more + (int)attn_quotient(grain - longer, line.each);
}

// Zeros for rows from, from + step, ... < to of q, by a warp: they see no key
// (`real`: of a request), or lie behind the last sequence.
__device__ __forceinline__ void attn_no_keys(const AttnArgs& p, int64_t from, int64_t to, int64_t step, bool real) {
  const int quads = p.a.D / 8, lane = threadIdx.x & 31;
  for (int64_t t = from; t < to; t += step) {
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.a.out) + t * p.a.out_row;
    for (int i = lane; i < p.a.Hq * quads; i += 32)
      *reinterpret_cast<uint4*>(out + (int64_t)(i / quads) * p.a.out_head + 8 * (i % quads)) = make_uint4(0, 0, 0, 0);
    if (p.a.lse)
      for (int h = lane; h < p.a.Hq; h += 32) p.a.lse[t * p.a.Hq + h] = real && p.a.sinks ? p.a.sinks[h] : -INFINITY;
  }
}

// The queries of a request that see no key: the first `before`, and those
// from `past` on.
struct AttnBlind {
  int before, past;
};
__device__ __forceinline__ AttnBlind attn_blind(const AttnArgs& p, const AttnRequest& q) {
  const int first = q.length - q.n;  // position of the first query
  if (p.capacity == 0) return {q.n, q.n};
  // (windows that lie behind the table)
  const int64_t past = p.a.window > 0 ? (int64_t)p.capacity + p.a.window - 1 - first : q.n;
  return {min(max(-first, 0), q.n), (int)max(min(past, (int64_t)q.n), (int64_t)0)};
}

// Every CTA finds the line's length and its worker's stretch [u, u_end) of
// it, or each of its warps' own (then `team` is 1; CTA 0 writes the line
// down); false where it has none.  Items that average fewer units than
// kTeamSpan go to warps (kTeams warps of a CTA can be workers).  A request's
// tiles are gone through by one thread, in every CTA: of a prompt of 131072
// tokens under a window of 128 (64 / 8 heads) that is some 8% of 3.2 ms.
template <int kRows, int kUnit, int kThreads, int kTeams, int kTeamSpan, int kWhole>
__device__ __forceinline__ bool attn_stretch(const AttnArgs& p, AttnCursor<kRows, kUnit, kWhole>& cursor, int64_t& u,
                                             int64_t& u_end, int& team) {
  constexpr int kWarps = kThreads / 32;
  __shared__ int64_t warp_units[kWarps], found_rest[kTeams];
  __shared__ int warp_items[kWarps], found[kTeams];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int each = ceil_div(max(p.a.R, 1), kThreads);
  const int r0 = min((int)threadIdx.x * each, p.a.R), r1 = min(r0 + each, p.a.R);
  const int start = p.a.R > 0 ? min(max(p.a.offsets[0], 0), p.a.T) : 0;
  const int end = p.a.R > 0 ? min(max(p.a.offsets[p.a.R], 0), p.a.T) : 0;
  int64_t mine = 0;
  int items = 0;
  bool blind = false;  // a request of this thread's has queries that see no key
  for (int r = r0; r < r1; ++r) {
    const AttnRequest q = attn_request(p, r);
    const int tiles = attn_tiles<kRows>(p, q);
    items += tiles * p.a.Hkv;
    int64_t sum = 0;
    for (int i = 0; i < tiles; ++i) sum += attn_span<kUnit>(p, q, i * kRows, kRows).units;
    mine += sum * p.a.Hkv;
    const AttnBlind b = attn_blind(p, q);
    blind = blind || b.before > 0 || b.past < q.n;
  }
  int64_t before = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, before, o);
    if (lane >= o) before += x;
  }
  items = __reduce_add_sync(0xffffffffu, items);
  if (lane == 31) warp_units[warp] = before, warp_items[warp] = items;
  before -= mine;
  __syncthreads();
  int64_t units = 0, all_items = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_units[w];
    units += warp_units[w];
    all_items += warp_items[w];
  }
  if (__any_sync(0xffffffffu, blind))
    for (int i = 0; i < each; ++i) {
      AttnRequest q = {0, 0, 0};
      AttnBlind b = {0, 0};
      if (r0 + i < r1) {
        q = attn_request(p, r0 + i);
        b = attn_blind(p, q);
      }
      for (unsigned todo = __ballot_sync(0xffffffffu, b.before > 0 || b.past < q.n); todo; todo &= todo - 1) {
        const int from = __ffs(todo) - 1;
        const int64_t row0 = __shfl_sync(0xffffffffu, q.row0, from), n = __shfl_sync(0xffffffffu, q.n, from);
        const int first = __shfl_sync(0xffffffffu, b.before, from), past = __shfl_sync(0xffffffffu, b.past, from);
        attn_no_keys(p, row0 + blockIdx.x, row0 + first, gridDim.x, true);
        attn_no_keys(p, row0 + past + blockIdx.x, row0 + n, gridDim.x, true);
      }
    }
  if (start > 0 || max(start, end) < p.a.T) {
    const int64_t at = (int64_t)blockIdx.x * kWarps + warp, step = (int64_t)gridDim.x * kWarps;
    attn_no_keys(p, at, start, step, false);
    attn_no_keys(p, max(start, end) + at, p.a.T, step, false);
  }

  team = kTeams > 1 && units < kTeamSpan * all_items ? 1 : kTeams;
  static_assert(kTeams == 1 || kTeams == 4, "a grain is a unit of each warp");
  const int most = team == kTeams ? p.workers / kTeams : p.workers;
  const int64_t worth = max(all_items, attn_quotient(units, p.least)), grains = kTeams > 1 && team > 1 ? (units + 3) / 4 : units;
  const AttnLine line = attn_line(units, (int)max(min((int64_t)most, min(worth, grains)), (int64_t)1),
                                  kTeams > 1 && team > 1 ? 2 : 0);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.line = line;
  const int teams = kTeams / team, w0 = (int)blockIdx.x * teams;
  if (line.units == 0 || w0 >= line.workers) return false;
  for (int i = 0; i < teams; ++i) {
    const int64_t at_u = w0 + i < line.workers ? attn_start(line, w0 + i) : 0;
    if (before <= at_u && at_u < before + mine) {
      int64_t at = before;
      int r = r0;
      for (; r + 1 < r1; ++r) {
        const int64_t n = attn_units<kRows, kUnit>(p, r);
        if (at_u < at + n) break;
        at += n;
      }
      found[i] = r;
      found_rest[i] = at_u - at;
    }
  }
  __syncthreads();
  const int i = team == 1 && kTeams > 1 ? warp : 0, w = w0 + i;
  u = u_end = 0;
  if (w >= line.workers) return true;
  u = attn_start(line, w);
  u_end = attn_start(line, w + 1);
  cursor.start(p, found[i], found_rest[i]);
  const bool passes = cursor.from > 0 && cursor.span.units <= kWhole;  // (an item that a worker before has whole)
  if (team == 1 && kTeams > 1 ? lane == 0 : threadIdx.x == 0)
    p.places[w] = {cursor.q.row0, cursor.q.length - cursor.q.n, cursor.tile, cursor.head, cursor.rows(p),
                   passes ? 0 : cursor.from, cursor.span.units};
  if (passes) {
    u += cursor.span.units - cursor.from;
    if (u < u_end) cursor.next(p);
  }
  return true;
}

// The next item of a cursor in shared memory, which is a warp's own.
template <int kRows, int kUnit, int kWhole>
__device__ __forceinline__ void attn_next(const AttnArgs& p, AttnCursor<kRows, kUnit, kWhole>& c) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) c.next(p);
  __syncwarp();
}

// The units of the cursor's item that are this worker's, of a stretch of `left`.
template <int kRows, int kUnit, int kWhole>
__device__ __forceinline__ int attn_take(const AttnCursor<kRows, kUnit, kWhole>& c, int64_t left) {
  return c.span.units <= kWhole ? c.span.units - c.from : (int)min((int64_t)c.span.units - c.from, left);
}

// ---------------------------------------------------------------- pieces of the kernels
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// A row's probabilities are 2^(x - m) in FP16 (x in units of log 2).  m moves
// when a score outgrows it by kMost, to kBelow below that score: they stay
// within FP16's 65504, and the largest is at least 2^kBelow, so that what FP16
// rounds below its normal range is off by 2^-25 beside that, 2^-32 of the
// largest.  (Against the largest itself, the many weak keys beside a strong one
// of zero value lost a quarter of their weight at 18 units of e below it.)  m
// lags by up to kMost - kBelow: with 8 chunks of 2048 tokens behind 8192 take
// 583 us, with 4, which moves the sums more often, 745.
constexpr float kBelow = 7.f, kMost = 15.f;

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

// The power of two that brings a row's largest |q| to [2^14, 2^15) (one below
// 2^-112 less far, as the power is an FP32 number), and its inverse.
__device__ __forceinline__ float row_scale(float top, float& back) {
  const int e = max((int)((__float_as_uint(top) >> 23) & 0xff) - 127 - 14, -126);
  back = __uint_as_float((uint32_t)(127 + e) << 23);
  return __uint_as_float((uint32_t)(127 - e) << 23);
}

// Whether a query at this position sees a key.
__device__ __forceinline__ bool attn_sees(const AttnArgs& p, int pos) {
  return pos >= 0 && (p.a.window == 0 || pos - p.a.window < p.capacity - 1);
}

// A row's last step: from its maximum (units of log 2) and divisor, with the
// sink's term, the factor of its sums, and its lse.  pos: its query's position.
__device__ __forceinline__ float attn_finish(const AttnArgs& p, int head, int pos, float top, float sum, float& lse) {
  if (top == -INFINITY && sum == 0.f) {  // no key, or scores of -inf: 0 / 0 without a sink
    lse = p.a.sinks ? p.a.sinks[head] : -INFINITY;
    return lse == -INFINITY && attn_sees(p, pos) ? NAN : 0.f;
  }
  float by = 1.f;
  if (p.a.sinks) {
    const float sink = p.a.sinks[head] * kLog2e, next = fmaxf(top, sink);
    if (sink == INFINITY && top < sink && sum == sum) {  // (all of the weight, and inf - inf below)
      lse = p.a.sinks[head];
      return 0.f;
    }
    if (next != -INFINITY) {
      by = top == -INFINITY ? 1.f : exp2_approx(top - next);  // (-inf: none but NaN scores)
      sum = sum * by + exp2_approx(sink - next);
      top = next;
    }
  }
  lse = (top == -INFINITY ? 0.f : top) * kLn2 + logf(sum);
  return p.a.v_scale * by / sum;
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

constexpr int kJoinThreads = 256, kJoinParts = 64;  // parts at a time

// The parts of the item that worker w's stretch begins in the middle of: w -
// 1's second place and the first ones of w .. last, summed in that order.
template <int D, int kRows, int kJoin>
__device__ __forceinline__ void attn_join(const AttnArgs& p, const AttnPlace& at, int row0, int w, int last) {
  // a thread has four columns of a row, kGroups threads the same, kTurns times
  constexpr int kQuads = D / 4;
  constexpr int kBusy = kJoin * kQuads < kJoinThreads ? kJoin * kQuads : kJoinThreads;
  constexpr int kGroups = kJoinThreads / kBusy, kTurns = kJoin * kQuads / kBusy;
  __shared__ float factor[kJoin][kJoinParts];
  __shared__ float old_factor[kJoin], tops[kJoin], sums[kJoin];
  __shared__ float4 shared_acc[kGroups > 1 ? kJoinThreads : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = min(at.rows - row0, kJoin);
  if (rows <= 0) return;
  const int parts = last - w + 2;
  auto part_of = [&](int x) { return 2 * (int64_t)(w - 1 + x) + (x == 0 ? 1 : 0); };
  __syncthreads();  // (the item before this one is done with what they share)
  float4 acc[kTurns];
#pragma unroll
  for (int y = 0; y < kTurns; ++y) acc[y] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (threadIdx.x < kJoin) tops[threadIdx.x] = -INFINITY, sums[threadIdx.x] = 0.f;
  for (int x0 = 0; x0 < parts; x0 += kJoinParts) {
    const int n = min(parts - x0, kJoinParts);
    __syncthreads();
    for (int row = warp; row < rows; row += kJoinThreads / 32) {
      float mx[kJoinParts / 32], lx[kJoinParts / 32];
      float top = tops[row];
      const float before = top;
#pragma unroll
      for (int y = 0; y < kJoinParts / 32; ++y) {
        const int x = lane + 32 * y;
        const float2 st = x < n ? *reinterpret_cast<const float2*>(attn_stats<D, kRows>(p, part_of(x0 + x), row0 + row))
                                : make_float2(-INFINITY, 0.f);
        mx[y] = st.x, lx[y] = st.y;
        top = fmaxf(top, st.x);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      float sum = 0.f;
#pragma unroll
      for (int y = 0; y < kJoinParts / 32; ++y) {
        // (equal: both may be -inf, of parts without a key, or of NaN scores)
        const float by = mx[y] == top ? 1.f : exp2_approx(mx[y] - top);
        factor[row][lane + 32 * y] = by;
        sum += lx[y] * by;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      __syncwarp();
      if (lane == 0) {
        const float by = before == top ? 1.f : exp2_approx(before - top);
        old_factor[row] = by;
        sums[row] = sums[row] * by + sum;
        tops[row] = top;
      }
    }
    __syncthreads();
#pragma unroll
    for (int y = 0; y < kTurns; ++y) {
      const int i = threadIdx.x % kBusy + y * kBusy, row = i / kQuads, d = 4 * (i % kQuads);
      if (row >= rows) continue;
      const float by = old_factor[row];
      acc[y].x *= by, acc[y].y *= by, acc[y].z *= by, acc[y].w *= by;
#pragma unroll 8
      for (int x = threadIdx.x / kBusy; x < n; x += kGroups) {
        const float4 v = *reinterpret_cast<const float4*>(p.parts + (part_of(x0 + x) * kRows + row0 + row) * D + d);
        const float f = factor[row][x];
        acc[y].x += v.x * f, acc[y].y += v.y * f, acc[y].z += v.z * f, acc[y].w += v.w * f;
      }
    }
  }
  if constexpr (kGroups > 1) {  // (one turn)
    shared_acc[threadIdx.x] = acc[0];
    __syncthreads();
    if (threadIdx.x >= kBusy) return;
#pragma unroll
    for (int y = 1; y < kGroups; ++y) {
      const float4 v = shared_acc[threadIdx.x + y * kBusy];
      acc[0].x += v.x, acc[0].y += v.y, acc[0].z += v.z, acc[0].w += v.w;
    }
  }
#pragma unroll
  for (int y = 0; y < kTurns; ++y) {
    const int i = threadIdx.x % kBusy + y * kBusy, row = i / kQuads, d = 4 * (i % kQuads);
    if (row >= rows) continue;
    const AttnRows r = attn_row(p, attn_rows(p, at.tile * kRows), row0 + row);
    const int token = at.row0 + r.query, hq = at.head * p.group + r.head;
    float lse;
    const float inv = attn_finish(p, hq, at.first + r.query, tops[row], sums[row], lse);
    *reinterpret_cast<uint2*>(attn_out(p, token, hq) + d) =
        make_uint2(pack_bf16x2(acc[y].x * inv, acc[y].y * inv), pack_bf16x2(acc[y].z * inv, acc[y].w * inv));
    if (p.a.lse && d == 0) p.a.lse[(int64_t)token * p.a.Hq + hq] = lse;
  }
}

// Joins each item that workers share, kJoin rows at a time, where the first
// stretch that begins in its middle does.  The CTAs look through their shares
// of workers and groups of rows, 32 at a time.
template <int D, int kRows, int kJoin>
__global__ void __launch_bounds__(kJoinThreads) attention_join_kernel(AttnArgs p) {
  constexpr int kGroupsOfRows = kRows / kJoin;
  pdl_wait();
  pdl_launch_dependents();
  const AttnLine line = *p.line;
  if (line.units == 0) return;
  const int all = line.workers * kGroupsOfRows;
  for (int i0 = blockIdx.x; i0 < all; i0 += 32 * gridDim.x) {
    const int mine = i0 + (threadIdx.x & 31) * (int)gridDim.x, worker = mine / kGroupsOfRows;
    bool joins = false;
    if (mine < all && worker > 0) {
      const int from = p.places[worker].from;
      joins = from != 0 && attn_start(line, worker - 1) <= attn_start(line, worker) - from;
    }
    for (unsigned todo = __ballot_sync(0xffffffffu, joins); todo; todo &= todo - 1) {
      const int i = i0 + (__ffs(todo) - 1) * (int)gridDim.x, w = i / kGroupsOfRows;
      const AttnPlace at = p.places[w];
      attn_join<D, kRows, kJoin>(p, at, (i % kGroupsOfRows) * kJoin, w,
                                 attn_owner(line, attn_start(line, w) - at.from + at.units - 1));
    }
  }
}

// Its CTAs, 4 and 8 an SM: with a quarter of them five queries of 16 requests
// of 16384 tokens take 102 us instead of 97, chunks of 2048 behind 8192 599
// instead of 580; with twice as many one request of 4096 13.2 instead of 12.2
// (and those 16 requests 93).
template <int D, int kRows, int kJoin>
cudaError_t launch_attention_join(const AttnArgs& p, int sms, cudaStream_t st) {
  const int grid = min(p.workers * (kRows / kJoin), (kRows > 16 ? 8 : 4) * sms);
  return launch_dependent(attention_join_kernel<D, kRows, kJoin>, (unsigned)grid, kJoinThreads, st, p);
}

}  // namespace moe_fp4
