// Attention over the paged cache of 4 bits (moe_fp4_attention): a few rows to
// a key head, as in decoding, and the join of what workers share.
//
//   x_j = scale k_scale q . k_j,  out = v_scale sum_j e^(x_j - m) v_j / sum_j e^(x_j - m)
//
// in one pass over the cache, against an m that follows the maximum (in units
// of log 2; kBelow, attention_work.cuh).
//
// Every warp streams blocks of 16 tokens of its own (keys and values of a head
// lie together: one bulk copy of 18 D bytes each) through a ring in shared
// memory, decodes them in registers (E2M1 by the hardware's conversion, times
// the E4M3 scale, exact in FP16) straight into the operands of
// mma.m16n8k16: the 16 tokens are the rows of K q^T, whose columns are the
// heads that share the key head, so that eight heads fill the product, and
// the columns of V^T p^T.  Between the two, p is a transposition away
// (movmatrix) from the second product's operand.  Tokens are dealt to the
// products' rows as (0, 4, 1, 5, 2, 6, 3, 7), and the same 8 later, so that
// the lanes that read the values of their two tokens at once lie on other
// banks.  q is scaled by a power of two per row into FP16's range.
//
// Bound by the cache's bytes (0.56 of a byte a value, each read once for a
// group of up to 16 rows) and by the 600 or so instructions that a warp takes
// for 32 tokens of 128 columns, which take as long: of 64 requests' 440 MB the
// copies alone take 76 us, the whole call 100 (4.4 TB/s), 8 of them the join of
// shared items (the counters: 57% of the issue slots, half of the ALU's, 52%
// of the memory's time).  Half of the instructions turn codes into FP16 and
// scale them: products of 8-bit operands would not carry a code times its
// scale exactly.
#include "attention_work.cuh"
#include "host.cuh"
#include "tcgen05.cuh"

namespace moe_fp4 {

static __device__ uint32_t g_attention_status;

cudaError_t attention_status_address(void** p) { return cudaGetSymbolAddress(p, g_attention_status); }

namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kPair = 2 * kCacheBlock;  // tokens that a warp takes in one go: two blocks
// Items of fewer pairs on average go to a warp each (windows of 128 tokens of
// 128 requests: 16.4 us; with the four warps of a CTA to an item 24.4).
constexpr int kTeamSpan = 64;
// Items of at most so many pairs are one worker's: a warp takes 0.6 us a pair by
// itself, a part and its join about 4 us (64 / 8 heads of 64, windows of 128:
// 16.3 us, with 3 pairs 22.1; 32 / 8 heads of 128, 64 requests of 300 tokens:
// 21.7 us, with 12 pairs 25.7, though 256 of them take 46 and 31).
constexpr int kWholePairs = 6;
// Pairs that are worth a worker, where there are workers to spare (32 / 8 heads
// of 128: 64 requests of 300 tokens 21.7 us, with 1 pair 23.5, with 8 26.2; one
// request of 300 13.4, 10.4, 16.8; one of 1000 12.6, 11.9, 15.5).
constexpr int kLeastPairs = 4;
constexpr uint32_t kWaitCode = 1u;

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// Two E4M3 scales as an FP16 pair.
__device__ __forceinline__ uint32_t scale_pair(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}

// The same with NaN as 448 (the minimum of a number and a NaN is the number).
__device__ __forceinline__ uint32_t finite_scale_pair(uint32_t two) {
  uint32_t r;
  asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(scale_pair(two)), "r"(0x5f005f00u));
  return r;
}

// The token of a block that row i of its 16 stands for.
__device__ __forceinline__ int row_token(int i) { return (i & 8) + ((i & 7) >> 1) + 4 * (i & 1); }

template <int D, int NT>
struct Cfg {
  static constexpr int kRows = 8 * NT;
  static constexpr int kStages = D == 256 ? 2 : 3;
  static constexpr int kStageBytes = 2 * cache_block_bytes(D);
  static constexpr int kRing = kStages * kStageBytes;  // a warp's
  static constexpr int kRow = D + 4;                   // floats of a row of sums (padded: rows start on other banks)
  static_assert(kRows * kRow * 4 <= kRing, "a warp's sums lie in its ring");
  static constexpr int kBarriers = kWarps * kStages * 8;
  static constexpr int kStats = kWarps * kRows * 2 * 4;
  static constexpr int kSmem = kWarps * kRing + kBarriers + kStats;
  static constexpr int kCtas = D * NT <= 128 ? 4 : D * NT <= 256 ? 3 : 2;  // per SM
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, Cfg<D, NT>::kCtas) attention_rows_kernel(AttnArgs p) {
  using C = Cfg<D, NT>;
  constexpr int kRows = C::kRows, S = C::kStages;
  constexpr int kSteps = D / 16;  // K steps of q . k, row tiles of V^T
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kWarps * C::kRing);
  float* stats = reinterpret_cast<float*>(smem + kWarps * C::kRing + C::kBarriers);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * C::kRing;
  uint64_t* full = bars + warp * S;

  if (lane == 0)
    for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
  fence_mbar_init();
  pdl_wait();
  pdl_launch_dependents();

  // each warp's place in its stretch (in shared memory: registers are worth more to the loop)
  __shared__ AttnCursor<kRows, kPair, kWholePairs> cursors[kWarps];
  AttnCursor<kRows, kPair, kWholePairs>& c = cursors[warp];
  int64_t u, u_end;
  int team;
  {
    AttnCursor<kRows, kPair, kWholePairs> start;
    if (!attn_stretch<kRows, kPair, kThreads, kWarps, kTeamSpan>(p, start, u, u_end, team)) return;
    if (lane == 0) c = start;
    __syncwarp();
  }
  const int member = team == 1 ? 0 : warp, worker = team == 1 ? (int)blockIdx.x * kWarps + warp : (int)blockIdx.x;

  const uint8_t* cache = static_cast<const uint8_t*>(p.a.cache);
  const int blocks_log = 31 - __clz(p.a.page_size / kCacheBlock);  // blocks of a page
  int stage = 0;  // that the next pair is read from, and its phase
  uint32_t phase = 0;
  bool alive = true;

  while (u < u_end) {
    const AttnRequest q = c.q;
    const AttnSpan span = c.span;
    const int r = c.r, tile = c.tile, head = c.head, from = c.from;
    const int to = from + attn_take(c, u_end - u);
    u += to - from;

    // this warp's pairs of blocks: first, first + team, ...; their copies
    // start before anything else
    const int end_block = (min((span.first + to) * kPair, span.hi) + kCacheBlock - 1) / kCacheBlock;
    const int first = span.first + from + member, end_pair = span.first + to;
    const int count = alive && first < end_pair ? (end_pair - first + team - 1) / team : 0;
    const int32_t* table = p.a.tables + (int64_t)r * p.a.table_row;
    // of 32 pairs at a time, a lane each: which block of the cache it is (memory
    // holds fewer than 2^32), the page of its odd block (pages of one block), and
    // which blocks' pages there are not
    uint32_t at_block = 0;
    int odd = 0;
    unsigned bad_even = 0, bad_odd = 0;
    unsigned bad_blocks = 0;  // of the copies in flight: two bits per stage
    auto load = [&](int i, int fill) {
      if ((i & 31) == 0) {
        const int b = 2 * (first + (i + lane) * team);
        int even = b < end_block ? table[b >> blocks_log] : 0;
        odd = blocks_log == 0 && b + 1 < end_block ? table[b + 1] : even;
        const bool bad0 = (unsigned)even >= (unsigned)p.a.pages, bad1 = (unsigned)odd >= (unsigned)p.a.pages;
        bad_even = __ballot_sync(0xffffffffu, bad0), bad_odd = __ballot_sync(0xffffffffu, bad1);
        even = bad0 ? 0 : even, odd = bad1 ? 0 : odd;
        at_block = (((uint32_t)even * p.a.Hkv + head) << blocks_log) + (b & ((1 << blocks_log) - 1));
      }
      if ((bad_even | bad_odd | bad_blocks) != 0)
        bad_blocks = (bad_blocks & ~(3u << (2 * fill))) |
                     (((bad_even >> (i & 31) & 1u) | (bad_odd >> (i & 31) & 1u) << 1) << (2 * fill));
      if (lane == (i & 31)) {
        uint8_t* dst = ring + fill * C::kStageBytes;
        const uint8_t* src = cache + (int64_t)at_block * cache_block_bytes(D);
        const int blocks = min(end_block - 2 * (first + i * team), 2);
        mbar_arrive_expect_tx(&full[fill], blocks * cache_block_bytes(D));
        if (blocks_log > 0) {  // the two lie together
          bulk_load(dst, src, blocks * cache_block_bytes(D), &full[fill]);
        } else {
          bulk_load(dst, src, cache_block_bytes(D), &full[fill]);
          if (blocks == 2)
            bulk_load(dst + cache_block_bytes(D), cache + ((int64_t)odd * p.a.Hkv + head) * cache_block_bytes(D),
                      cache_block_bytes(D), &full[fill]);
        }
      }
    };
    for (int i = 0; i < min(S - 1, count); ++i) load(i, stage + i < S ? stage + i : stage + i - S);

    // q, in the operand's order, and the rows' factors
    uint32_t qf[NT][kSteps][2];
    float fac[NT][2];
    int last[NT][2];  // position of the columns' queries, -1: no row
    const int base_pos = q.length - q.n;
    const int rows = c.rows(p);
    const AttnRows tile_rows = attn_rows(p, tile * kRows);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const AttnRows row = attn_row(p, tile_rows, 8 * n + g);
      float v[D / 4], top = 0.f;
      const bool real = 8 * n + g < rows;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.a.q) + (int64_t)(q.row0 + row.query) * p.a.q_row +
                                 (int64_t)(head * p.group + row.head) * p.a.q_head + t * (D / 4);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const uint4 w = real ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0, 0, 0, 0);
        const uint32_t b[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[8 * i + 2 * j] = __uint_as_float(b[j] << 16);
          v[8 * i + 2 * j + 1] = __uint_as_float(b[j] & 0xffff0000u);
        }
      }
#pragma unroll
      for (int i = 0; i < D / 4; ++i) top = fmaxf(top, fabsf(v[i]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      float back;
      const float by = row_scale(top, back);
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        qf[n][j][0] = pack_f16x2(v[4 * j] * by, v[4 * j + 1] * by);
        qf[n][j][1] = pack_f16x2(v[4 * j + 2] * by, v[4 * j + 3] * by);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        fac[n][c] = __shfl_sync(0xffffffffu, back, 4 * (2 * t + c)) * (p.a.scale * p.a.k_scale * kLog2e);
        const int col = 8 * n + 2 * t + c;
        last[n][c] = col < rows ? base_pos + attn_row(p, tile_rows, col).query : -1;
      }
    }
    // blocks that every row sees whole
    const int pos_first = base_pos + tile_rows.query;
    const int pos_last = base_pos + attn_row(p, tile_rows, rows - 1).query;
    const int all_lo = p.a.window > 0 ? max(pos_last - p.a.window + 1, 0) : 0;

    float o[NT][kSteps][4], m[NT][2], minus[NT][2], l[NT][2];  // (minus: -m, or 0 while that is -inf)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < kSteps; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
      m[n][0] = m[n][1] = -INFINITY;
      minus[n][0] = minus[n][1] = 0.f;
      l[n][0] = l[n][1] = 0.f;
    }

    for (int i = 0; i < count; ++i) {
      if (i + S - 1 < count) load(i + S - 1, stage == 0 ? S - 1 : stage - 1);  // (the stage of pair i - 1)
      if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase, &g_attention_status, kWaitCode))) {
        // (the other copies on their way end before the CTA does)
        for (int x = i + 1; x < min(i + S, count); ++x) {
          if (++stage == S) stage = 0, phase ^= 1;
          mbar_wait(&full[stage], phase, &g_attention_status, kWaitCode);
        }
        alive = false;
        break;
      }
      const uint8_t* at = ring + stage * C::kStageBytes;
      const int tok0 = (first + i * team) * kPair;

      // S^T = K q^T: rows g, g + 8 of each block
      float s[2][NT][4];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int n = 0; n < NT; ++n) s[b][n][0] = s[b][n][1] = s[b][n][2] = s[b][n][3] = 0.f;
        const uint8_t* kb = at + b * cache_block_bytes(D);
        constexpr int kWords = D / 32;  // words of codes per lane and row
        uint32_t w[2][kWords];
        uint32_t by[2][(kWords + 1) / 2];  // a scale for two words, in both halves
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int tok = row_token(g + 8 * h);
          const uint8_t* row = kb + tok * (D / 2) + t * (D / 8);
          if constexpr (D == 64) {
            const uint2 x = *reinterpret_cast<const uint2*>(row);
            w[h][0] = x.x, w[h][1] = x.y;
          } else {
#pragma unroll
            for (int j = 0; j < kWords; j += 4) {
              const uint4 x = *reinterpret_cast<const uint4*>(row + 4 * j);
              w[h][j] = x.x, w[h][j + 1] = x.y, w[h][j + 2] = x.z, w[h][j + 3] = x.w;
            }
          }
          const uint8_t* sr = kb + 8 * D + tok * (D / 16) + t * (D / 64);
          if constexpr (D == 64) {
            by[h][0] = __byte_perm(scale_pair(*sr), 0, 0x1010);
          } else {
#pragma unroll
            for (int j = 0; j < D / 64; j += 2) {
              const uint32_t two = scale_pair(*reinterpret_cast<const uint16_t*>(sr + j));
              by[h][j] = __byte_perm(two, 0, 0x1010);
              by[h][j + 1] = __byte_perm(two, 0, 0x3232);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          uint32_t x[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            e2m1x8_to_half2x4(w[h][j], x[h]);
#pragma unroll
            for (int k = 0; k < 4; ++k) x[h][k] = mul_f16x2(x[h][k], by[h][j / 2]);
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t af[4] = {x[0][2 * k], x[1][2 * k], x[0][2 * k + 1], x[1][2 * k + 1]};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(s[b][n], af, qf[n][2 * j + k][0], qf[n][2 * j + k][1]);
          }
        }
      }

      // scores in units of log 2, masked (an item's last pair may reach past the
      // end of a table that is shorter than its request, so that it always is
      // masked: a bound of its own spills, two requests of 262144 tokens 103 us
      // for 101.5)
      const bool whole = tok0 >= all_lo && tok0 + kPair - 1 <= pos_first && (i + 1 < count || to < span.units);
      const unsigned bad = (bad_blocks >> (2 * stage)) & 3u;
      bool grows = false;
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[b][n][e] *= fac[n][e & 1];
      if (!whole || bad != 0) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = tok0 + kCacheBlock * b + row_token(g + 8 * (e >> 1)), pos = last[n][e & 1];
              if (bad >> b & 1u) s[b][n][e] = NAN;
              // (a table ends at a block's end)
              if (tok0 + kCacheBlock * b >= p.capacity || !(j <= pos && (p.a.window == 0 || j > pos - p.a.window)))
                s[b][n][e] = -INFINITY;
            }
      }
      // m follows when a score outgrows it by 2^kMost
      float top[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2) {
          top[n][c2] = fmaxf(fmaxf(s[0][n][c2], s[0][n][c2 + 2]), fmaxf(s[1][n][c2], s[1][n][c2 + 2]));
          grows = grows || top[n][c2] > m[n][c2] + kMost;
        }
      if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int c2 = 0; c2 < 2; ++c2) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) top[n][c2] = fmaxf(top[n][c2], __shfl_xor_sync(0xffffffffu, top[n][c2], x));
            const float next = fmaxf(m[n][c2], top[n][c2] - kBelow);
            const float by = next == -INFINITY ? 1.f : exp2_approx(m[n][c2] - next);
            m[n][c2] = next;
            minus[n][c2] = next == -INFINITY ? 0.f : -next;
            l[n][c2] *= by;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
              o[n][j][c2] *= by;
              o[n][j][c2 + 2] *= by;
            }
          }
        }
      }
      uint32_t pf[2][NT][2];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float e[4];
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            e[i4] = exp2_approx(s[b][n][i4] + minus[n][i4 & 1]);
            l[n][i4 & 1] += e[i4];
          }
          pf[b][n][0] = transpose8x8(pack_f16x2(e[0], e[1]));
          pf[b][n][1] = transpose8x8(pack_f16x2(e[2], e[3]));
        }

      // O^T += V^T p^T: columns g D / 8 .. of the values, tokens t, t + 4, t + 8, t + 12 of each block
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const uint8_t* vb = at + b * cache_block_bytes(D) + cache_half_bytes(D);
        constexpr int kWords = D / 64;  // words of codes per lane and token
        uint32_t w[4][kWords];
        uint32_t sc[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint8_t* row = vb + (t + 4 * k) * (D / 2) + g * (D / 16);
          const uint8_t* sr = vb + 8 * D + (t + 4 * k) * (D / 16) + g * (D / 8) / 16;
          if constexpr (D == 64) {
            w[k][0] = *reinterpret_cast<const uint32_t*>(row);
            sc[k] = *sr;
          } else if constexpr (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2*>(row);
            w[k][0] = x.x, w[k][1] = x.y;
            sc[k] = *sr;
          } else {
            const uint4 x = *reinterpret_cast<const uint4*>(row);
            w[k][0] = x.x, w[k][1] = x.y, w[k][2] = x.z, w[k][3] = x.w;
            sc[k] = *reinterpret_cast<const uint16_t*>(sr);
          }
        }
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
          uint32_t x[4][4];  // rows of even and odd columns, tokens (t, t + 4); the same, tokens (t + 8, t + 12)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t a = w[2 * k][j], bb = w[2 * k + 1][j];
            const uint32_t even = (a & 0x0f0f0f0fu) | ((bb & 0x0f0f0f0fu) << 4);
            const uint32_t odd = ((a >> 4) & 0x0f0f0f0fu) | (bb & 0xf0f0f0f0u);
            const uint32_t by = finite_scale_pair(__byte_perm(sc[2 * k], sc[2 * k + 1], j < 2 ? 0x40 : 0x51));
            e2m1x8_to_half2x4(even, x[2 * k]);
            e2m1x8_to_half2x4(odd, x[2 * k + 1]);
#pragma unroll
            for (int i4 = 0; i4 < 4; ++i4) {
              x[2 * k][i4] = mul_f16x2(x[2 * k][i4], by);
              x[2 * k + 1][i4] = mul_f16x2(x[2 * k + 1][i4], by);
            }
          }
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            const uint32_t af[4] = {x[0][i4], x[1][i4], x[2][i4], x[3][i4]};
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16(o[n][4 * j + i4], af, pf[b][n][0], pf[b][n][1]);
          }
        }
      }
      __syncwarp();  // the pair is read: its stage may be loaded anew
      if (++stage == S) stage = 0, phase ^= 1;
    }

    // the warps' sums, joined
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) l[n][c] += __shfl_xor_sync(0xffffffffu, l[n][c], x);
    const bool is_whole = from == 0 && to == span.units;
    const int64_t part = 2 * (int64_t)worker + (from == 0 ? 1 : 0);
    if (team == 1) {
      // a lane has D / 8 columns of the heads 2 t, 2 t + 1
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2) {
          const int row = 8 * n + 2 * t + c2;
          if (row >= rows) continue;
          if (!is_whole) {
            float* dst = p.parts + (part * kRows + row) * D + g * (D / 8);
#pragma unroll
            for (int j = 0; j < kSteps; j += 2)
              *reinterpret_cast<float4*>(dst + 2 * j) = make_float4(o[n][j][c2], o[n][j][c2 + 2], o[n][j + 1][c2], o[n][j + 1][c2 + 2]);
            if (g == 0) *reinterpret_cast<float2*>(attn_stats<D, kRows>(p, part, row)) = make_float2(m[n][c2], l[n][c2]);
            continue;
          }
          const AttnRows rr = attn_row(p, tile_rows, row);
          const int token = q.row0 + rr.query, hq = head * p.group + rr.head;
          float lse;
          const float inv = attn_finish(p, hq, base_pos + rr.query, m[n][c2], l[n][c2], lse);
          __nv_bfloat16* dst = attn_out(p, token, hq) + g * (D / 8);
#pragma unroll
          for (int j = 0; j < kSteps; j += 4)
            *reinterpret_cast<uint4*>(dst + 2 * j) =
                make_uint4(pack_bf16x2(o[n][j][c2] * inv, o[n][j][c2 + 2] * inv),
                           pack_bf16x2(o[n][j + 1][c2] * inv, o[n][j + 1][c2 + 2] * inv),
                           pack_bf16x2(o[n][j + 2][c2] * inv, o[n][j + 2][c2 + 2] * inv),
                           pack_bf16x2(o[n][j + 3][c2] * inv, o[n][j + 3][c2 + 2] * inv));
          if (p.a.lse && g == 0) p.a.lse[(int64_t)token * p.a.Hq + hq] = lse;
        }
      __syncwarp();
      if (u < u_end) attn_next(p, c);
      continue;
    }
    float* sums = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float* row = sums + (8 * n + 2 * t + c) * C::kRow + g * (D / 8);
#pragma unroll
        for (int j = 0; j < kSteps; ++j) *reinterpret_cast<float2*>(row + 2 * j) = make_float2(o[n][j][c], o[n][j][c + 2]);
        if (g == 0) {
          stats[(warp * kRows + 8 * n + 2 * t + c) * 2] = m[n][c];
          stats[(warp * kRows + 8 * n + 2 * t + c) * 2 + 1] = l[n][c];
        }
      }
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * (D / 4); i += kThreads) {
      const int row = i / (D / 4), d = 4 * (i % (D / 4));
      if (row >= rows) break;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stats[(w * kRows + row) * 2]);
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = stats[(w * kRows + row) * 2];
        const float by = mw == -INFINITY ? (top == -INFINITY ? 1.f : 0.f) : exp2_approx(mw - top);
        // (a warp whose maximum is -inf has sums of zero, or NaN from NaN scores)
        const float lw = stats[(w * kRows + row) * 2 + 1];
        const float4 v = *reinterpret_cast<const float4*>(smem + w * C::kRing + (row * C::kRow + d) * 4);
        sum += lw * by;
        acc.x += v.x * by;
        acc.y += v.y * by;
        acc.z += v.z * by;
        acc.w += v.w * by;
      }
      if (!is_whole) {
        *reinterpret_cast<float4*>(p.parts + (part * kRows + row) * D + d) = acc;
        if (d == 0) *reinterpret_cast<float2*>(attn_stats<D, kRows>(p, part, row)) = make_float2(top, sum);
        continue;
      }
      const AttnRows rr = attn_row(p, tile_rows, row);
      const int token = q.row0 + rr.query, hq = head * p.group + rr.head;
      float lse;
      const float inv = attn_finish(p, hq, base_pos + rr.query, top, sum, lse);
      *reinterpret_cast<uint2*>(attn_out(p, token, hq) + d) =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (p.a.lse && d == 0) p.a.lse[(int64_t)token * p.a.Hq + hq] = lse;
    }
    fence_proxy_async_smem();  // the sums lie where the next copies go
    __syncthreads();
    if (u < u_end) attn_next(p, c);
  }
}

int max_ctas(int sms, int D, int NT) { return sms * (D * NT <= 128 ? 4 : D * NT <= 256 ? 3 : 2); }

template <int D, int NT>
cudaError_t launch_rows(AttnArgs p, int sms, cudaStream_t st) {
  using C = Cfg<D, NT>;
  static bool seen[64];
  cudaError_t e = allow_smem(attention_rows_kernel<D, NT>, C::kSmem, seen);
  if (e != cudaSuccess) return e;
  const int grid = max_ctas(sms, D, NT);
  p.workers = grid * kWarps;
  p.least = kLeastPairs;
  e = launch_dependent_smem(attention_rows_kernel<D, NT>, (unsigned)grid, kThreads, C::kSmem, st, p);
  if (e != cudaSuccess) return e;
  // few items: many parts to each, joined by more CTAs (one request of 4096
  // tokens 12.0 us, by eight rows 14.5; 64 requests 99, by two rows 110)
  const int64_t tiles = p.a.R > 0 ? ((int64_t)p.a.T * p.group / p.a.R + C::kRows - 1) / C::kRows : 0;
  return p.a.R * tiles * p.a.Hkv <= 64 ? launch_attention_join<D, C::kRows, 2>(p, sms, st)
                                       : launch_attention_join<D, C::kRows, 8>(p, sms, st);
}

template <int D>
cudaError_t launch_dim(const AttnArgs& p, int sms, cudaStream_t st) {
  // Rows that an average request has to a key head: up to 8 fill one product of
  // 8 columns, up to 16 two, more go to tiles of 128.  16 requests of 16384
  // tokens, 8 key heads of 128, us:
  //   rows                      4     8    12    16    20    32    48    64
  //   one product, again       65    66   113   113
  //   two products, again      85    86    87    88   156   157   223   291
  //   tiles                   174   175   175   176   176   176   180   181
  // (From 17 to 32 rows tiles take a tenth longer at these sizes, 81 for 67 with
  // 64 requests of 1000 tokens, 157 for 102 with heads of 64.)  It is
  // one kernel for a call, by the mean over all requests and with rows of q
  // behind the last sequence: requests of other kinds in a batch are served by
  // the wrong one (63 single tokens behind 8192 and a chunk of 2048, 32 / 8
  // heads: 643 us, 112 and 236 apart; 255 and a chunk of 512: 842, 406 and 91;
  // 64 single tokens 113, padded to 256 rows 155).
  const int64_t rows = p.a.R > 0 ? (int64_t)p.a.T * p.group / p.a.R : 0;
  if (rows > 16) return launch_attention_tc(p, (int)rows, sms, st);
  return rows > 8 ? launch_rows<D, 2>(p, sms, st) : launch_rows<D, 1>(p, sms, st);
}

constexpr int kMaxWorkers = 4 * kWarps;  // per SM
size_t places_bytes(int sms) { return ((size_t)sms * kMaxWorkers * sizeof(AttnPlace) + 255) / 256 * 256; }

}  // namespace

size_t attention_workspace_bytes(int, int, int, int D) {
  int sms = 0;
  if (current_device_sms(&sms) != cudaSuccess) sms = 152;
  size_t parts = attention_tc_parts_bytes(D, sms);
  for (int NT = 1; NT <= 2; ++NT) {
    const size_t n = (size_t)2 * max_ctas(sms, D, NT) * kWarps * 8 * NT * (D + 2) * 4;
    parts = n > parts ? n : parts;
  }
  return 256 + places_bytes(sms) + (parts + 255) / 256 * 256;
}

cudaError_t launch_attention(const moe_fp4_attention_args& a, cudaStream_t st) {
  int sms = 0;
  const cudaError_t e = current_device_sms(&sms);
  if (e != cudaSuccess) return e;
  AttnArgs p = {};
  p.a = a;
  p.group = a.Hq / a.Hkv;
  p.inverse = (65536 + p.group - 1) / p.group;
  p.capacity = a.table_width * a.page_size;
  p.line = static_cast<AttnLine*>(a.workspace);
  p.places = reinterpret_cast<AttnPlace*>(static_cast<char*>(a.workspace) + 256);
  p.parts = reinterpret_cast<float*>(static_cast<char*>(a.workspace) + 256 + places_bytes(sms));
  switch (a.D) {
    case 64: return launch_dim<64>(p, sms, st);
    case 128: return launch_dim<128>(p, sms, st);
    default: return launch_dim<256>(p, sms, st);
  }
}

}  // namespace moe_fp4
