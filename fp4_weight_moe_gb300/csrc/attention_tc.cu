// Attention over the paged cache of 4 bits for many rows to a key head
// (prompts and their chunks), on the 5th-generation tensor cores (sm_103a).
//
// A CTA takes kTiles tiles of 128 rows (query and head of a group each) over a
// key head's tokens, kTok at a time (a step):
//   softmax warps  (four or eight per tile of rows) own a row, or half of its
//                  columns, per thread: they bring q to shared memory as FP16,
//                  scaled by a power of two per row; read a step's scores from
//                  tensor memory, follow their maximum, and put p =
//                  2^(x - m) back over them in FP16, the second product's A
//                  operand; at the end they read the sums and write the rows;
//   decode warps   turn the cache's codes into FP16 (exact: at most six
//                  significant bits in [2^-10, 2688]) in shared memory, in the
//                  128-byte-swizzled layout that the products read: keys
//                  K-major, values as they lie, N-major;
//   MMA warp       converged, issues S = Q K^T into tensor memory and O += P V
//                  (P from tensor memory) as their operands come;
//   load warp      a block's half (keys or values of 16 tokens) to a bulk
//                  copy, a lane each, into a ring of half steps.
// With two tiles each has its scores; while one's softmax runs, the other's
// products do.  With one (few rows, or D = 256, whose sums take half of tensor
// memory) two buffers of scores alternate between steps.
//
// Bound, with two tiles, by the chain of a tile's softmax (2100 cycles for 128
// tokens: 640 instructions a warp, between waits on tensor memory) and its two
// products (1090), of which two tiles hide one another's in part: the tensor
// cores are busy 47% of the time (chunks of 2048 tokens behind 8192, 32 query
// heads, D = 128: 580 us, 1.07 PFLOP/s).  With one tile by what a step hands
// over from one to the next, whatever number of its rows is real: 16 requests of
// 16384 tokens (32 / 8 heads of 128, 302 MB) take 176 us with 20 rows and 186
// with 128, 3400 cycles a step.  Left out, the decoding (141 us), the softmax
// (158), the copies (168), all three (120) show that none of them is the bound:
// the last is the products, 590 cycles each, and their signals, in turn.
//
// m follows the scores only when they outgrow it by 2^kMost, to 2^kBelow below
// them (p stays within FP16, sums and divisor are taken against the same m), so
// that the sums in tensor memory are hardly ever rescaled.
#include "attention_work.cuh"
#include "gemm_f16w4.cuh"
#include "gemm_fp8.cuh"

namespace moe_fp4 {

namespace {

// Items of at most so many steps are one worker's (40 rows, 32 / 8 heads of 128:
// 64 requests of 200 tokens 42.1 us, with 1 step 45.2; 8 requests of 1000 24.0,
// with 8 steps 25.3; in between 64 of 300 tokens would take 47 with 4, not 56),
// and steps that are worth a worker (8 requests of 1000 tokens 24.0 us, with 1
// step 28.8, with 8 24.8; one of 16384 38.7, 38.7, 29.2).
constexpr int kWholeSteps = 2, kLeastSteps = 4;

template <int D, int kTiles_>
struct TcCfg {
  static constexpr int kTiles = kTiles_;
  static constexpr int kRows = 128 * kTiles;
  static constexpr int kTok = D <= 128 ? 128 : 64;
  static constexpr int kBlocks = kTok / kCacheBlock;
  static constexpr uint32_t kQTile = 128 * D * 2;
  static constexpr uint32_t kKv = kTok * D * 2;  // decoded keys or values of a step
  static constexpr uint32_t kPanel = kTok * 128;    // 64 columns of them: swizzled rows of 128 bytes
  static constexpr uint32_t kHalf = kBlocks * cache_half_bytes(D);
  static constexpr int kRaw = D == 64 || (D == 128 && kTiles == 1) ? 6 : 3;  // half steps in flight
  // A row's threads: two with one tile, which has no other tile's products to
  // hide its softmax (35 rows of five requests of up to 100000 tokens 273 us with
  // one, 257 with two); two tiles have, and twice the warps take more
  // instructions (chunks of 2048 tokens 586 us with one, 611 with two).
  static constexpr int kSides = kTiles == 1 ? 2 : 1;
  static constexpr int kCols = kTok / kSides;  // of a step's scores: a softmax thread's
  static constexpr int kSoftWarps = 4 * kSides * kTiles;
  static constexpr int kDecWarps = 8;
  static constexpr int kMmaWarp = kSoftWarps + kDecWarps, kLoadWarp = kMmaWarp + 1;
  static constexpr int kThreads = 32 * (kMmaWarp + 4);  // (whole warpgroups, for the split of registers)
  // registers of the softmax, the decode and the last warpgroup's threads: together no more than the launch's
  static constexpr int kSoftRegs = 136, kDecRegs = 72, kLastRegs = 64;
  static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;
  static_assert(32 * (kSoftWarps * kSoftRegs + kDecWarps * kDecRegs + 4 * kLastRegs) <= kThreads * kLaunchRegs, "registers");
  static constexpr uint32_t kTmemO = 2 * 128;    // the sums lie behind two buffers of scores
  // the sums go out by way of 4096 bytes to a softmax warp: the queries' place, if that is enough
  static constexpr uint32_t kStage = D == 64 && kSides == 2 ? 4096 * kSoftWarps : 0;
  static constexpr uint32_t kBytes = kTiles * kQTile + 4 * kKv + kRaw * kHalf + kStage;
  static constexpr uint32_t kBarBytes = 512;
  static constexpr uint32_t kSmem = kBytes + kBarBytes + 1024 /*align*/;
  static_assert(kSmem <= 227 * 1024, "shared memory");
  static_assert(kTmemO + kTiles * D <= 512, "tensor memory");
};

// The low word of an operand's shared-memory descriptor (its address; offsets
// in units of 16 bytes add to it), and the high words of the two kinds: rows
// of 128 bytes along K, eight to a swizzled group of 1024 bytes; and, for the
// values, rows along N, with `lbo` (in the low word) to the next 64 of N.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return (uint32_t)smem_desc(saddr, lbo, 1024, kLayoutSW128);
}
__device__ __forceinline__ uint32_t desc_hi() { return (uint32_t)(smem_desc(0, 16, 1024, kLayoutSW128) >> 32); }

// Four K = 16 steps of D (+)= A B from a converged warp, operands kA and kB
// units of 16 bytes apart from step to step; the first adds to D if `add`.
template <int kA, int kB>
__device__ __forceinline__ void mma_f16_4(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q, e;\n\t.reg .b64 da, db;\n\t.reg .b32 ta, tb;\n\t"
      "setp.ne.u32 p, %5, 0;\n\tsetp.eq.u32 q, %4, %4;\n\telect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t"
      "add.u32 ta, %1, %6;\n\tadd.u32 tb, %2, %7;\n\tmov.b64 da, {ta, %3};\n\tmov.b64 db, {tb, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, q;\n\t"
      "add.u32 ta, ta, %6;\n\tadd.u32 tb, tb, %7;\n\tmov.b64 da, {ta, %3};\n\tmov.b64 db, {tb, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, q;\n\t"
      "add.u32 ta, ta, %6;\n\tadd.u32 tb, tb, %7;\n\tmov.b64 da, {ta, %3};\n\tmov.b64 db, {tb, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, q;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(add ? 1u : 0u), "n"(kA), "n"(kB)
      : "memory");
}

// The same with A (FP16, a row per lane, two values a column) in tensor memory.
template <int kB>
__device__ __forceinline__ void mma_f16_ts_4(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q, e;\n\t.reg .b64 db;\n\t.reg .b32 ta, tb;\n\t"
      "setp.ne.u32 p, %5, 0;\n\tsetp.eq.u32 q, %4, %4;\n\telect.sync _|e, 0xffffffff;\n\t"
      "mov.b64 db, {%2, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t"
      "add.u32 ta, %1, 8;\n\tadd.u32 tb, %2, %6;\n\tmov.b64 db, {tb, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %4, q;\n\t"
      "add.u32 ta, ta, 8;\n\tadd.u32 tb, tb, %6;\n\tmov.b64 db, {tb, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %4, q;\n\t"
      "add.u32 ta, ta, 8;\n\tadd.u32 tb, tb, %6;\n\tmov.b64 db, {tb, %3};\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [ta], db, %4, q;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(add ? 1u : 0u), "n"(kB)
      : "memory");
}

__device__ __forceinline__ float2 fadd2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\tmov.b64 ra, {%2,%3};\n\tmov.b64 rb, {%4,%5};\n\t"
      "add.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0,%1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// The warps that share rows (one, or two of 64 threads, all of which come):
// whether any of them says so.
template <int kSides>
__device__ __forceinline__ bool rows_any(int id, bool x) {
  if constexpr (kSides == 1) return __any_sync(0xffffffffu, x);
  uint32_t r;
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.or.pred q, %1, 64, p;\n\t"
               "selp.u32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"(id), "r"((uint32_t)x) : "memory");
  return r != 0;
}
template <int kSides>
__device__ __forceinline__ void rows_sync(int id) {
  if constexpr (kSides == 1)
    __syncwarp();
  else
    asm volatile("barrier.cta.sync %0, 64;" ::"r"(id) : "memory");
}

constexpr uint32_t kTcWait = 2u;

template <int D, int kTiles>
__global__ void __launch_bounds__(TcCfg<D, kTiles>::kThreads, 1) attention_tc_kernel(AttnArgs p, uint32_t* err) {
  using C = TcCfg<D, kTiles>;
  constexpr int kTok = C::kTok, kSides = C::kSides;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* q_smem = smem;
  uint8_t* k_smem = q_smem + kTiles * C::kQTile;  // two buffers
  uint8_t* v_smem = k_smem + 2 * C::kKv;          // two buffers
  uint8_t* raw = v_smem + 2 * C::kKv;
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(raw + C::kRaw * C::kHalf + C::kStage);
  uint64_t* raw_empty = raw_full + C::kRaw;
  uint64_t* kv_full = raw_empty + C::kRaw;  // [keys 0, keys 1, values 0, values 1]
  uint64_t* kv_empty = kv_full + 4;
  uint64_t* s_full = kv_empty + 4;  // [2] scores of a buffer are there
  uint64_t* p_full = s_full + 2;    // [2] probabilities are
  uint64_t* pv_done = p_full + 2;   // [2] sums of a tile are
  uint64_t* q_full = pv_done + 2;   // [2] a tile's queries are there, and its sums read
  uint64_t* item_done = q_full + 2;  // all sums of an item are (with one tile)
  uint32_t* bad_blocks = reinterpret_cast<uint32_t*>(item_done + 1);  // [kRaw]
  uint32_t* tmem_slot = bad_blocks + C::kRaw;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kRaw; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], C::kDecWarps);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&kv_full[i], C::kDecWarps);
      mbar_init(&kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4 * C::kSides);
      mbar_init(&pv_done[i], 1);
      mbar_init(&q_full[i], 4 * C::kSides);
    }
    mbar_init(item_done, 1);
    fence_mbar_init();
  }
  pdl_wait();
  pdl_launch_dependents();
  // each warp's place in its CTA's stretch (in shared memory: its registers
  // are worth more to the loops between items)
  __shared__ AttnCursor<C::kRows, kTok, kWholeSteps> cursors[C::kThreads / 32];
  AttnCursor<C::kRows, kTok, kWholeSteps>& c = cursors[warp];
  // what the threads of a row tell each other: its queries' factor (in the
  // first half), their scores' largest, their divisors
  __shared__ float told[2][C::kRows];
  __shared__ uint32_t dead[4 * kTiles];  // a wait of a row's gave up
  __shared__ float far_fac[32 * C::kSoftWarps];  // of threads whose scores are large: their factor
  if (threadIdx.x < 4 * kTiles) dead[threadIdx.x] = 0;  // (seen behind the barrier below)
  int left;  // units of the stretch that are left
  {
    int64_t u, u_end;
    int team;
    AttnCursor<C::kRows, kTok, kWholeSteps> start;
    if (!attn_stretch<C::kRows, kTok, C::kThreads, 1, 0>(p, start, u, u_end, team)) return;
    if (lane == 0) c = start;
    __syncwarp();
    left = (int)(u_end - u);
  }

  if (warp == C::kMmaWarp) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity & 1, err, kTcWait));
  };

  if (warp >= C::kSoftWarps + C::kDecWarps) {
    regs_dec<C::kLastRegs>();
    if (warp == C::kLoadWarp) {
      const uint8_t* cache = static_cast<const uint8_t*>(p.a.cache);
      const int blocks_log = 31 - __clz(p.a.page_size / kCacheBlock);
      uint32_t half = 0;
      bool ok = true;
      while (ok && left > 0) {
        const int steps = attn_take(c, left);
        const int end_block = (c.span.hi + kCacheBlock - 1) / kCacheBlock;
        const int32_t* table = p.a.tables + (int64_t)c.r * p.a.table_row;
        int b = (c.span.first + c.from) * C::kBlocks + lane;
        auto page_of = [&](int block) { return lane < C::kBlocks && block < end_block ? table[block >> blocks_log] : 0; };
        int page = page_of(b);
        for (int i = 0; i < steps; ++i, b += C::kBlocks) {
          const bool mine = lane < C::kBlocks && b < end_block;
          const bool bad = mine && (page < 0 || page >= p.a.pages);
          const int64_t at = ((((int64_t)(bad ? 0 : page) * p.a.Hkv + c.head) << blocks_log) + (b & ((1 << blocks_log) - 1))) *
                             cache_block_bytes(D);
          const unsigned real = __ballot_sync(0xffffffffu, mine), wrong = __ballot_sync(0xffffffffu, bad);
          page = i + 1 < steps ? page_of(b + C::kBlocks) : 0;
          for (int kind = 0; ok && kind < 2; ++kind, ++half) {
            const uint32_t s = half % C::kRaw, round = half / C::kRaw;
            if (round > 0 && !wait(&raw_empty[s], round - 1)) {
              ok = false;
              break;
            }
            if (lane == 0) {
              bad_blocks[s] = wrong;
              mbar_arrive_expect_tx(&raw_full[s], __popc(real) * cache_half_bytes(D));
            }
            __syncwarp();
            if (mine)
              bulk_load(raw + s * C::kHalf + lane * cache_half_bytes(D), cache + at + kind * cache_half_bytes(D),
                        cache_half_bytes(D), &raw_full[s]);
          }
          if (!ok) break;
        }
        left -= steps;
        if (left > 0) attn_next(p, c);
      }
      // (whoever gave up: the copies on their way end before the CTA does)
      for (uint32_t h = half > C::kRaw ? half - C::kRaw : 0; h < half; ++h) wait(&raw_full[h % C::kRaw], h / C::kRaw);
    } else if (warp == C::kMmaWarp) {
      const uint32_t idesc_s = idesc_f16(128, kTok), idesc_o = idesc_f16(128, D) | (1u << 16);
      uint32_t step = 0;         // over all items
      uint32_t item = 0;
      bool ok = true;
      const uint32_t hi = desc_hi();
      const uint32_t q_lo = desc_lo(smem_u32(q_smem), 16), k_lo = desc_lo(smem_u32(k_smem), 16);
      const uint32_t v_lo = desc_lo(smem_u32(v_smem), C::kPanel);
      auto scores = [&](int tile, uint32_t at, int buffer) {  // S = Q K^T of step `at` into a buffer
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < D / 64; ++k)  // 64 columns: a panel
          mma_f16_4<2, 2>(tmem + buffer * 128, q_lo + tile * (C::kQTile >> 4) + k * 1024,
                          k_lo + (at & 1) * (C::kKv >> 4) + k * (C::kPanel >> 4), hi, idesc_s, k > 0);
        mma_commit_warp(&s_full[buffer]);
      };
      auto sums = [&](int tile, uint32_t at, int buffer, bool first) {  // O += P V
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kTok / 64; ++k)  // 16 tokens a step: 2048 bytes
          mma_f16_ts_4<128>(tmem + C::kTmemO + tile * D, tmem + buffer * 128 + 32 * k,
                            v_lo + (at & 1) * (C::kKv >> 4) + k * 512, hi, idesc_o, !first || k > 0);
        mma_commit_warp(&pv_done[tile]);
      };
      uint32_t p_seen[2] = {0, 0};
      while (ok && left > 0) {
        const int steps = attn_take(c, left);
        if constexpr (kTiles == 2) {
          ok = wait(&kv_full[step & 1], step >> 1);
          for (int n = 0; ok && n < 2; ++n) {
            ok = wait(&q_full[n], item);
            if (ok) scores(n, step, n);
          }
          if (!ok) break;
          mma_commit_warp(&kv_empty[step & 1]);
          for (int i = 0; ok && i < steps; ++i, ++step) {
            const uint32_t next = step + 1;
            for (int n = 0; ok && n < 2; ++n) {
              ok = wait(&p_full[n], p_seen[n]++);
              if (ok && n == 0) ok = wait(&kv_full[2 + (step & 1)], step >> 1);
              if (!ok) break;
              sums(n, step, n, i == 0);
              if (n == 1) mma_commit_warp(&kv_empty[2 + (step & 1)]);
              if (i + 1 < steps) {
                if (n == 0) ok = wait(&kv_full[next & 1], next >> 1);
                if (!ok) break;
                scores(n, next, n);
                if (n == 1) mma_commit_warp(&kv_empty[next & 1]);
              }
            }
          }
        } else {
          ok = wait(&q_full[0], item);
          for (int j = 0; ok && j < min(steps, 2); ++j) {
            const uint32_t at = step + j;
            ok = wait(&kv_full[at & 1], at >> 1);
            if (!ok) break;
            scores(0, at, at & 1);
            mma_commit_warp(&kv_empty[at & 1]);
          }
          for (int i = 0; ok && i < steps; ++i, ++step) {
            const int buffer = step & 1;
            ok = wait(&p_full[buffer], p_seen[buffer]++);
            if (ok) ok = wait(&kv_full[2 + (step & 1)], step >> 1);
            if (!ok) break;
            sums(0, step, buffer, i == 0);
            if (i + 1 == steps) mma_commit_warp(item_done);
            mma_commit_warp(&kv_empty[2 + (step & 1)]);
            if (i + 2 < steps) {
              const uint32_t at = step + 2;
              ok = wait(&kv_full[at & 1], at >> 1);
              if (!ok) break;
              scores(0, at, at & 1);
              mma_commit_warp(&kv_empty[at & 1]);
            }
          }
        }
        ++item;
        left -= steps;
        if (ok && left > 0) attn_next(p, c);
      }
    }
  } else if (warp >= C::kSoftWarps) {
    // decode: a unit is 32 values of a token
    regs_dec<C::kDecRegs>();
    constexpr int kParts = D / 32, kDecThreads = 32 * C::kDecWarps;
    const int tid = threadIdx.x - 32 * C::kSoftWarps;
    // a thread's units are kDecThreads / kParts tokens apart, a multiple of 16:
    // the same place in other blocks
    constexpr int kApart = kDecThreads / kParts;
    static_assert(kApart % 16 == 0 && kTok % kApart == 0, "units");
    const int tok = tid / kParts, part = tid % kParts;
    // its chunks in an order that puts a quarter warp's on banks of their own
    const int turn = D == 64 ? 0 : D == 128 ? 2 * (part / 2) : part / 2;
    const int from = (tok / 16) * cache_half_bytes(D) + (tok % 16) * (D / 2) + part * 16;
    const int scales = (tok / 16) * cache_half_bytes(D) + 8 * D + (tok % 16) * (D / 16) + part * 2;
    const uint32_t first = turn & 2 ? 0x3232 : 0x1010;
    const int to = (part / 2) * C::kPanel + tok * 128, chunk = (4 * (part % 2)) ^ turn ^ (tok & 7);
    uint32_t s = 0, phase = 0, half = 0;
    bool ok = true;
    while (ok && left > 0) {
      const int steps = attn_take(c, left);
      for (int i = 0; ok && i < 2 * steps; ++i, ++half) {
        const uint32_t step = half >> 1, kind = half & 1, buf = 2 * kind + (step & 1), round = step >> 1;
        ok = wait(&raw_full[s], phase);
        if (ok && round > 0) ok = wait(&kv_empty[buf], round - 1);
        if (!ok) break;
        const uint8_t* src = raw + s * C::kHalf;
        uint8_t* dst = (kind ? v_smem : k_smem) + (step & 1) * C::kKv + to;
        const uint32_t wrong = kind ? 0 : bad_blocks[s] >> (tok / 16);
#pragma unroll
        for (int x = 0; x < kTok / kApart; ++x) {
          const uint8_t* block = src + x * (kApart / 16) * cache_half_bytes(D);
          uint2 a = *reinterpret_cast<const uint2*>(block + from + (turn & 2 ? 8 : 0));
          uint2 b = *reinterpret_cast<const uint2*>(block + from + (turn & 2 ? 0 : 8));
          uint32_t sb = *reinterpret_cast<const uint16_t*>(block + scales);
          if (wrong >> (x * (kApart / 16)) & 1u) sb = 0x7f7fu;
          uint32_t s2;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"((uint16_t)sb));
          if (kind) asm("min.f16x2 %0, %0, %1;" : "+r"(s2) : "r"(0x5f005f00u));  // (a value's NaN scale counts as 448)
          const uint32_t s0 = __byte_perm(s2, s2, first), s1 = __byte_perm(s2, s2, first ^ 0x2222);
          if (turn & 1) a = make_uint2(a.y, a.x), b = make_uint2(b.y, b.x);
          uint8_t* row = dst + x * kApart * 128;
          *reinterpret_cast<uint4*>(row + ((chunk ^ 0) << 4)) = e2m1x8_scaled_f16(a.x, s0);
          *reinterpret_cast<uint4*>(row + ((chunk ^ 1) << 4)) = e2m1x8_scaled_f16(a.y, s0);
          *reinterpret_cast<uint4*>(row + ((chunk ^ 2) << 4)) = e2m1x8_scaled_f16(b.x, s1);
          *reinterpret_cast<uint4*>(row + ((chunk ^ 3) << 4)) = e2m1x8_scaled_f16(b.y, s1);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&raw_empty[s]);
          mbar_arrive(&kv_full[buf]);
        }
        if (++s == C::kRaw) s = 0, phase ^= 1;
      }
      left -= steps;
      if (ok && left > 0) attn_next(p, c);
    }
  } else {
    regs_inc<C::kSoftRegs>();
    // a row's threads have kCols of a step's columns each, and D / kSides of the sums'
    const int n = warp / (4 * kSides), side_of = kSides == 2 ? (warp >> 2) & 1 : 0;
    const int row_in_tile = threadIdx.x & 127, tile_row = 128 * n + row_in_tile;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_tmem = tmem + lanes + C::kTmemO + n * D + side_of * (D / kSides);
    const int pair = 4 * n + (warp & 3), id = 1 + pair;  // (of the two warps that share rows: a barrier of their own)
    const int col0 = side_of * C::kCols;
    uint32_t step = 0;  // over all items
    uint32_t item = 0;
    bool ok = true;
    while (ok && left > 0) {
      const int steps = attn_take(c, left);
      float fac;
      const AttnRows tile_rows = attn_rows(p, c.tile * C::kRows);
      {
        const int rows = c.rows(p);
        // q in FP16, the sign of the scale with it: D / 8 lanes to a row, 32 / kSides of the rows to a warp
        constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kTurns = 32 / kSides / kAtOnce, kFlight = kTurns < 8 ? kTurns : 8;
        const int l = lane % kLanes, side = lane / kLanes, first = 32 * (warp & 3) + 32 / kSides * side_of;  // (row of the tile)
        float back = 1.f;
        uint8_t* dst = q_smem + n * C::kQTile + (l / 8) * 16384;
#pragma unroll 1
        for (int i = 0; i < kTurns; i += kFlight) {
          uint4 x[kFlight];
#pragma unroll
          for (int y = 0; y < kFlight; ++y) {
            const int r = 128 * n + first + (i + y) * kAtOnce + side;
            const AttnRows rr = attn_row(p, tile_rows, r);
            x[y] = r < rows ? *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.a.q) +
                                                              (int64_t)(c.q.row0 + rr.query) * p.a.q_row +
                                                              (int64_t)(c.head * p.group + rr.head) * p.a.q_head + 8 * l)
                            : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int y = 0; y < kFlight; ++y) {
            const int r = first + (i + y) * kAtOnce + side;
            float v[8], top = 0.f, b;
            bf16x8_to_float(x[y], v);
#pragma unroll
            for (int z = 0; z < 8; ++z) top = fmaxf(top, fabsf(v[z]));
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            float by = row_scale(top, b);
            by = p.a.scale < 0.f ? -by : p.a.scale == 0.f ? 0.f : by;
            *reinterpret_cast<uint4*>(dst + r * 128 + (((l % 8) ^ (r & 7)) << 4)) =
                make_uint4(pack_f16x2(v[0] * by, v[1] * by), pack_f16x2(v[2] * by, v[3] * by),
                           pack_f16x2(v[4] * by, v[5] * by), pack_f16x2(v[6] * by, v[7] * by));
            if (kSides == 2) {
              if (l == 0) told[0][128 * n + r] = b;
            } else {
              const float mine = __shfl_sync(0xffffffffu, b, (lane % kAtOnce) * kLanes);
              if (lane / kAtOnce == i + y) back = mine;
            }
          }
        }
        fence_proxy_async_smem();
        if (kSides == 2) {
          rows_sync<kSides>(id);
          back = told[0][tile_row];
        }
        fac = fmaxf(back * fabsf(p.a.scale) * p.a.k_scale * kLog2e, 0x1p-120f);  // (above 0: masked scores stay -inf)
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[n]);
      }
      int pos, lowest;          // the row's position, the first token that it sees
      int whole_lo, whole_hi;   // tokens that every row of the tile sees (none past the table, as in the masks)
      {
        const int rows = c.rows(p), base_pos = c.q.length - c.q.n;
        pos = tile_row < rows ? base_pos + attn_row(p, tile_rows, tile_row).query : -1;
        lowest = p.a.window > 0 ? max(max(pos, 0) - p.a.window + 1, 0) : 0;
        const int pos_last = base_pos + attn_row(p, tile_rows, min(128 * n + 128, rows) - 1).query;
        whole_lo = p.a.window > 0 ? max(max(pos_last, 0) - p.a.window + 1, 0) : 0;
        whole_hi = min(base_pos + attn_row(p, tile_rows, 128 * n).query, p.capacity - 1);
      }

      const int warp_rows = c.rows(p);
      float m = -INFINITY;
      float2 l = make_float2(0.f, 0.f);
      int tok0 = (c.span.first + c.from) * kTok;
      for (int i = 0; i < steps; ++i, ++step, tok0 += kTok) {
        const int buffer = kTiles == 2 ? n : (int)(step & 1);
        if (!wait(&s_full[buffer], kTiles == 2 ? step : step >> 1)) {
          if (kSides == 1 || tile_row - lane >= warp_rows) {
            ok = false;
            break;
          }
          dead[pair] = 1;  // (told before the next vote, behind which both warps leave)
        }
        tc_fence_after();
        if (tile_row - lane >= warp_rows) {  // (no rows of this warp's: nobody reads what it leaves)
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[buffer]);
          continue;
        }
        const uint32_t s_tmem = tmem + lanes + buffer * 128 + col0;
        if (tok0 < whole_lo || tok0 + kTok - 1 > whole_hi) {
          // masked where they are, so that the loop below has no test for it
          // (as predicates there, they took as many instructions as the rest)
          const int hi = min(pos, p.capacity - 1) - tok0 - col0, lo = lowest - tok0 - col0;
          const float by = whole_lo == INT_MAX ? far_fac[threadIdx.x] : 1.f;
#pragma unroll 1
          for (int x = 0; x < C::kCols; x += 16) {
            uint32_t s[16];
            tmem_ld16(s_tmem + x, s);
#pragma unroll
            for (int y = 0; y < 16; ++y)
              s[y] = x + y > hi || x + y < lo ? 0xff800000u : __float_as_uint(__fmul_rn(__uint_as_float(s[y]), by));
            tmem_st16(s_tmem + x, s);
          }
          tmem_wait_st();
        }
        uint32_t h[C::kCols / 2];
        float2 sum[2];  // (sums and maxima in chains of their own, which depend on one another less)
        // against the maximum so far; where a score outgrows it, once more against its own
#pragma unroll 1
        for (int pass = 0;; ++pass) {
          const float from_m = m == -INFINITY ? 0.f : m;
          const float2 fac2 = make_float2(fac, fac), minus = make_float2(-from_m, -from_m);
          float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          sum[0] = sum[1] = make_float2(0.f, 0.f);
          uint32_t s[2][16];
          TmemLd<16>::start(s_tmem, s[0]);
#pragma unroll
          for (int x = 0; x < C::kCols / 16; ++x) {
            TmemLd<16>::wait(s[x & 1]);
            if (x + 1 < C::kCols / 16) TmemLd<16>::start(s_tmem + 16 * (x + 1), s[(x + 1) & 1]);
#pragma unroll
            for (int y = 0; y < 16; y += 2)
              tops[y / 2 % 4] = max3(tops[y / 2 % 4], __uint_as_float(s[x & 1][y]), __uint_as_float(s[x & 1][y + 1]));
#pragma unroll
            for (int y = 0; y < 8; ++y) {
              float2 e = ffma2(make_float2(__uint_as_float(s[x & 1][2 * y]), __uint_as_float(s[x & 1][2 * y + 1])), fac2, minus);
              e.x = exp2_approx(e.x);
              e.y = exp2_approx(e.y);
              sum[y & 1] = fadd2(sum[y & 1], e);
              h[8 * x + y] = pack_f16x2(e.x, e.y);
            }
          }
          float top = max3(fmaxf(tops[0], tops[1]), tops[2], tops[3]) * fac;
          // (m -inf: as soon as there is a key; and behind it both have read their scores, over which p goes)
          if (kSides == 2) tc_fence_before();
          bool grows = top > m + kMost;
          const bool any = rows_any<kSides>(id, grows);
          if (kSides == 2) tc_fence_after();
          if (!any || pass > 0) break;
          if (kSides == 2) {
            told[side_of][tile_row] = top;
            rows_sync<kSides>(id);
            top = fmaxf(told[0][tile_row], told[1][tile_row]);
            grows = top > m + kMost;
          }
          const float next = grows ? top - kBelow : m, by = grows ? exp2_approx(m - next) : 1.f;
          m = next;
          l.x *= by;
          l.y *= by;
          // Where a unit of m, a rounded product, is no small number, the others
          // have to be rounded before m is taken away, too (fused, the largest's
          // distance would be anything): from here on they are, where they lie.
          if (__any_sync(0xffffffffu, fabsf(m) > 0x1p20f && m != -INFINITY) && whole_lo != INT_MAX) {
#pragma unroll 1
            for (int x = 0; x < C::kCols; x += 16) {
              uint32_t s[16];
              tmem_ld16(s_tmem + x, s);
#pragma unroll
              for (int y = 0; y < 16; ++y) s[y] = __float_as_uint(__fmul_rn(__uint_as_float(s[y]), fac));
              tmem_st16(s_tmem + x, s);
            }
            tmem_wait_st();
            far_fac[threadIdx.x] = fac;
            fac = 1.f;
            whole_lo = INT_MAX;
          }
          if (i > 0) {
            if (!wait(&pv_done[n], step - 1)) {
              ok = kSides == 2;
              if (kSides == 1) break;
              dead[pair] = 1;
            }
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < D / kSides / 16; ++x) {
              uint32_t o[16];
              tmem_ld16(o_tmem + 16 * x, o);
#pragma unroll
              for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * by);
              tmem_st16(o_tmem + 16 * x, o);
            }
          }
        }
        if (kSides == 1 && !ok) break;
        l = fadd2(l, fadd2(sum[0], sum[1]));
#pragma unroll
        for (int x = 0; x < C::kCols / 32; ++x)
          tmem_st16(s_tmem - col0 / 2 + 16 * x, *reinterpret_cast<uint32_t(*)[16]>(&h[16 * x]));
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buffer]);
        if (kSides == 2 && *(volatile uint32_t*)&dead[pair]) {
          ok = false;
          break;
        }
      }
      // (With one tile the last scores come before the last two sums.  Of those
      // neither can be waited for by its phase: a wait for the last is met by the
      // one two before it, and one for the last but one is not met once the last
      // is done too.  So an item has a barrier of its own.)
      if (kSides == 1) {
        if (!ok || !wait(&pv_done[n], step - 1)) break;
      } else {
        if (ok) ok = wait(item_done, item);
        told[side_of][tile_row] = l.x + l.y;
        if (rows_any<kSides>(id, !ok)) break;
      }
      tc_fence_after();
      // The sums go out by way of the queries' place (the item's scores are
      // all done): 128 bytes of a row at a time, so that stores lie along rows.
      const int rows = c.rows(p);
      const float sum = kSides == 1 ? l.x + l.y : told[0][tile_row] + told[1][tile_row];
      const bool whole = c.from == 0 && steps == c.span.units;
      const int64_t part = 2 * (int64_t)blockIdx.x + (c.from == 0 ? 1 : 0);
      float inv = 1.f;
      if (tile_row < rows) {
        if (whole) {
          const AttnRows rr = attn_row(p, tile_rows, tile_row);
          const int hq = c.head * p.group + rr.head;
          float lse;
          inv = attn_finish(p, hq, pos, m, sum, lse);
          if (p.a.lse && side_of == 0) p.a.lse[(int64_t)(c.q.row0 + rr.query) * p.a.Hq + hq] = lse;
        } else if (side_of == 0) {
          *reinterpret_cast<float2*>(attn_stats<D, C::kRows>(p, part, tile_row)) = make_float2(m, sum);
        }
      }
      uint8_t* stage = C::kStage ? raw + C::kRaw * C::kHalf + 4096 * warp  // 32 rows of 128 bytes, the warp's own
                                 : q_smem + n * C::kQTile + side_of * 16384 + (warp & 3) * 32 * 128;
      const int chunk_row = lane / 8, chunk = lane % 8, row0 = 128 * n + 32 * (warp & 3);
      const int row_bytes = (whole ? 2 : 4) * D / kSides;  // this warp's of a row
      uint8_t* to[8];  // where the lane's rows go
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        const int r = row0 + 4 * y + chunk_row;
        const AttnRows rr = attn_row(p, tile_rows, r);
        to[y] = r >= rows ? nullptr
                          : (whole ? reinterpret_cast<uint8_t*>(attn_out(p, c.q.row0 + rr.query, c.head * p.group + rr.head))
                                   : reinterpret_cast<uint8_t*>(p.parts + (part * C::kRows + r) * D)) +
                                side_of * row_bytes + 16 * chunk;
      }
#pragma unroll 1
      for (int x = 0; x < row_bytes; x += 128) {
        uint32_t o[32];
        if (whole) {
          constexpr int kLoads = D / kSides < 64 ? 1 : 2;  // (columns that make 128 bytes, or all that there are)
          uint32_t f[kLoads][32];
#pragma unroll
          for (int y = 0; y < kLoads; ++y) TmemLd<32>::start(o_tmem + x / 2 + 32 * y, f[y]);
#pragma unroll
          for (int y = 0; y < kLoads; ++y) TmemLd<32>::wait(f[y]);
#pragma unroll
          for (int z = 0; z < 16 * kLoads; ++z)
            o[z] = pack_bf16x2(__uint_as_float(f[z / 16][2 * z % 32]) * inv, __uint_as_float(f[z / 16][2 * z % 32 + 1]) * inv);
        } else {
          tmem_ld32(o_tmem + x / 4, o);
        }
        __syncwarp();
#pragma unroll
        for (int y = 0; y < 8; ++y)
          if (D / kSides >= 64 || 16 * y < row_bytes)
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((y ^ (lane & 7)) << 4)) =
                make_uint4(o[4 * y], o[4 * y + 1], o[4 * y + 2], o[4 * y + 3]);
        __syncwarp();
        uint4 v[8];
#pragma unroll
        for (int y = 0; y < 8; ++y)
          v[y] = *reinterpret_cast<const uint4*>(stage + (4 * y + chunk_row) * 128 + ((chunk ^ ((4 * y + chunk_row) & 7)) << 4));
#pragma unroll
        for (int y = 0; y < 8; ++y)
          if (to[y] && (D / kSides >= 64 || x + 16 * chunk < row_bytes)) *reinterpret_cast<uint4*>(to[y] + x) = v[y];
        __syncwarp();
      }
      if (kSides == 2) rows_sync<kSides>(id);  // (the next queries go over both sides' place)
      ++item;
      left -= steps;
      if (left > 0) attn_next(p, c);
    }
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (warp == C::kMmaWarp) tmem_dealloc(tmem, 512);
}

template <int D, int kTiles>
cudaError_t launch_tiles(AttnArgs p, int sms, cudaStream_t st) {
  using C = TcCfg<D, kTiles>;
  static bool seen[64];
  cudaError_t e = allow_smem(attention_tc_kernel<D, kTiles>, C::kSmem, seen);
  if (e != cudaSuccess) return e;
  void* err = nullptr;
  e = attention_status_address(&err);
  if (e != cudaSuccess) return e;
  p.workers = sms;
  p.least = kLeastSteps;
  e = launch_dependent_smem(attention_tc_kernel<D, kTiles>, (unsigned)sms, C::kThreads, C::kSmem, st, p, static_cast<uint32_t*>(err));
  if (e != cudaSuccess) return e;
  return launch_attention_join<D, C::kRows, 8>(p, sms, st);
}

// Tiles of rows side by side: two, but where D = 256 leaves room for the sums
// of one, and where an average request has rows for one (16 requests of 16384
// tokens, 32 / 8 heads of 128: 128 rows 186 us on one, 230 on two; 160 rows 336
// and 244; 2 requests of 4096, 256 rows: 37.5 and 31.4).
constexpr int most_tiles(int D) { return D <= 128 ? 2 : 1; }

template <int D>
cudaError_t launch_tc_dim(const AttnArgs& p, int rows, int sms, cudaStream_t st) {
  return rows <= 128 ? launch_tiles<D, 1>(p, sms, st) : launch_tiles<D, most_tiles(D)>(p, sms, st);
}

}  // namespace

size_t attention_tc_parts_bytes(int D, int sms) { return (size_t)2 * sms * 128 * most_tiles(D) * (D + 2) * 4; }

cudaError_t launch_attention_tc(const AttnArgs& p, int rows, int sms, cudaStream_t st) {
  switch (p.a.D) {
    case 64: return launch_tc_dim<64>(p, rows, sms, st);
    case 128: return launch_tc_dim<128>(p, rows, sms, st);
    default: return launch_tc_dim<256>(p, rows, sms, st);
  }
}

}  // namespace moe_fp4
