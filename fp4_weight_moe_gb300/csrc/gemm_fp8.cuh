// E4M3 x E4M3 products with FP32 scales per block of 128 on the
// 5th-generation tensor cores (sm_103a):
//   D[m][n] = sum_b sx[m][b] sw[n / 128][b] sum_{k in b} X[m][k] W[n][k],
// b the 128-K blocks, X and W E4M3 (K-major rows), the inner sums in tensor
// memory (tcgen05.mma kind::f8f6f4), the outer one in FP32 registers: a
// scale per 128 K cannot ride on the MMA (its block scales are powers of
// two per 32 K), so every K block gets an accumulator of its own, which the
// scale warps read, scale and add up while the next block multiplies.
//
// A CTA computes 128 x BN tiles in turn:
//   warp 0 lane 0  TMA producer: per K block the 128-row box (128 x 128 B)
//                  and the BN-row box, SWIZZLE_128B, into a ring;
//   warps 1, 2     (warp 1 allocates tensor memory) converged, issue the four
//                  K = 32 MMAs of a block into accumulator g % kAcc (each
//                  warp every second block), then the commits that publish
//                  the accumulator and free the stage;
//   warp 3         copies the scales of 16 K blocks at a time to shared
//                  memory (cp.async, any strides), a chunk ahead, across tile
//                  boundaries too;
//   scale warps    each reads its 32 accumulator lanes (and its half of the
//                  columns where BN >= 128), adds them, scaled, into
//                  registers, and stores the finished tile.  They hold as
//                  little else as they can: with the scales' copies among
//                  their work the compiler spilled inside their loop.
//
// The 128-row operand is X (kSwap = false) or W (kSwap = true: few tokens,
// the tokens on the MMA's N side).
//
// What bounds a 128 x 256 tile, in cycles per K block, each measured alone:
// the MMAs take 512; shared memory moves 128 bytes a cycle, and the MMAs read
// 48 KB of it and the loads write as much: 768; the scale warps' sums take 270
// (330 with their tensor-memory loads).  In the whole kernel a block takes
// about 800 (M=4096 K=N=7168, six waves of tiles: 144-151 us, 2.9 PFLOP/s; K=7168
// N=4096, four waves, the last a third full: 95-99 us, 2.5).  CTA pairs
// (cta_group::2, 256 x 256 tiles, 64 KB a block and SM) shorten the second
// bound to 512, but their hand-overs cross SMs: 118 us where this kernel then
// took 110, and no better with 192, 160 or 128 columns and up to three
// accumulators.
//
// Few tokens are bound by the chain of one CTA (launch and barriers, the first
// loads, its K blocks, the cluster's sums).  With the weights in L2, and with
// weights from memory, as a model's layers find theirs: M=1 K=7168 N=4096 7.0
// and 8.8 us for 29 MB (3.3 TB/s of HBM), M=64 10.1 and 11.3, M=64 K=2048 N=7168
// 7.7 and 8.7.
#pragma once

#include "common.cuh"
#include "fp8_quant.cuh"
#include "tcgen05.cuh"

namespace moe_fp4 {

constexpr int kF8BM = 128;
constexpr int kF8BK = 128;     // K elements (= bytes) per stage: one scale block

struct Fp8Args {
  const float* xs;  // activation scales, xs[m * xs_row + b * xs_blk]
  int64_t xs_row, xs_blk;
  int xs_vec;  // rows lie next to each other, four at a time in 16 bytes (M rounded up to that)
  const uint16_t* xb;  // kXq: the BF16 activations, xb[m * xb_row + k], in place of E4M3 ones and xs
  int64_t xb_row;
  const float* ws;  // weight scales, ws[(n / 128) * ws_row + b]
  int64_t ws_row;
  const __nv_bfloat16* add;  // added to the product before its rounding (or null)
  int64_t add_row;
  void* out;
  int64_t out_row;
  int out_f32;
  int early;  // the first weight loads may run before the launch before this one is complete
  int pairs;  // out rows start at a pair of values' boundary
  int vec;  // out (and add) rows start 16-byte aligned; 2: out's 32-byte
  int M, N, K;
};

// kTwo: shared memory and tensor memory for two CTAs per SM.  kXq > 0: the
// kernel quantises its tokens, into kXq K blocks of their own.
template <int BN, bool kSwap, bool kTwo = false, int kXq = 0>
struct F8Cfg {
  static constexpr bool kFuse = kXq > 0;
  // K blocks of scales per shared-memory chunk (kXq: all of the CTA's), and
  // the chunks (four of four blocks, M=4096 K=7168 N=4096: 100 us, not 96)
  static constexpr int kChunk = kFuse ? kXq : 16, kChunks = kFuse ? 1 : 2;
  static_assert(!kFuse || kSwap, "the kernel quantises a few tokens only");
  static constexpr int kHalves = BN >= 128 ? 2 : 1;
  static constexpr int kCols = BN / kHalves;  // accumulator columns per scale thread
  static constexpr int kLd = kCols / 2 < 32 ? kCols / 2 : 32;  // ... per tensor-memory load (an even count of them)
  static constexpr int kScaleWarps = 4 * kHalves;
  // 256 columns: 128 sums per scale thread and two loads in flight need more
  // registers than an even split of the SM's gives twelve warps, so the scale
  // warps take them (setmaxnreg) from the warpgroup of warps 0 .. 3
  static constexpr bool kMoveRegs = BN >= 256;
  // two warps issue MMAs, each into its own accumulators, so that the waits
  // and the issue of one hide behind the other's MMAs
  static constexpr int kMmaWarps = 2;
  static constexpr int kFirst = 2 + kMmaWarps;  // first scale warp
  static constexpr int kQuantWarps = kFuse ? 4 : 0;  // they help the scale warps quantise, then leave
  static constexpr int kThreads = 32 * (kFirst + kScaleWarps + kQuantWarps);
  static constexpr int kAcc = BN >= 256 ? 2 : 4;
  static constexpr uint32_t kTmemCols = kAcc * BN < 32 ? 32 : kAcc * BN;
  static constexpr int kXRows = kSwap ? BN : kF8BM;  // activation rows of a tile
  static constexpr int kWRows = kSwap ? kF8BM : BN;
  static constexpr int kWBlocks = kWRows / 128 < 1 ? 1 : kWRows / 128;
  static constexpr uint32_t kStageA = kF8BM * kF8BK;
  static constexpr uint32_t kStageB = kFuse ? 0 : BN * kF8BK;
  // eight rows per K block (one swizzle group); the MMA's rows 8 .. 15 read
  // into the block after, and so past the last one
  static constexpr uint32_t kXqBytes = kXq > 0 ? (kXq + 1) * 1024 : 0;
  static_assert(kXq == 0 || BN == 16, "at most eight tokens");
  static constexpr uint32_t kStageBytes = kStageA + kStageB;
  static constexpr uint32_t kScaleBytes = kChunks * kChunk * (kXRows + kWBlocks) * 4;
  static constexpr uint32_t kBarBytes = 256;
  // a scale warp's 32 x 16 values on their way to rows that allow no vector
  // stores (a word of padding, so that lanes at their own rows spread over the
  // banks)
  static constexpr int kOutRow = 17;
  static constexpr uint32_t kOutBytes = kSwap ? 0 : kScaleWarps * 32 * kOutRow * 4;
  static constexpr uint32_t kBudget =
      (kTwo ? 113u : 227u) * 1024u - 1024u - kBarBytes - kScaleBytes - kXqBytes - kOutBytes;
  // A multiple of the MMA warps, so that a stage's rounds are all one warp's: a
  // wait for a round's parity is also met two rounds earlier, and only a warp
  // that has waited for the round between cannot be early.
  static constexpr int kFit = kBudget / kStageBytes > 12 ? 12 : (int)(kBudget / kStageBytes);
  static constexpr int kStages = kFit / kMmaWarps * kMmaWarps;
  static constexpr uint32_t kSmem =
      kStages * kStageBytes + kXqBytes + kScaleBytes + kBarBytes + kOutBytes + 1024 /*align*/;
  static_assert(kTmemCols <= 512 && (kTmemCols & (kTmemCols - 1)) == 0, "tensor memory");
  static_assert(kAcc % kMmaWarps == 0, "an accumulator's uses, too, are one warp's");
  static_assert(kStages >= 4 && kSmem <= (kTwo ? 113 : 227) * 1024, "shared memory");
  static_assert(!kTwo || kTmemCols <= 256, "tensor memory of two CTAs");
  // a split tile's partial sums lie in the ring: [BN][128] tokens by columns
  // (kSwap) or [128][BN + 4] (padded, so that lanes writing their own rows
  // spread over the banks)
  static constexpr uint32_t kPartRow = kSwap ? 128 : BN + 4;
  static_assert(BN > 128 || (kSwap ? BN : 128) * kPartRow * 4u <= kStages * kStageBytes, "partial sums fit the ring");
  static_assert((2 * kStages + 2 * kAcc + 2 * kChunks + 1) * 8 + 4 <= (int)kBarBytes, "barrier block");
};

// Instruction descriptor of tcgen05.mma kind::f8f6f4: E4M3 A and B (format
// 0), both K-major, FP32 accumulator (format 1), M x N tile.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The four K = 32 MMAs of a K block (the first overwrites the accumulator)
// and the commits behind them, from one elected lane of a converged warp:
// `done` and `empty` are arrived on when the MMAs are complete.
__device__ __forceinline__ void mma_f8_block(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint64_t* done, uint64_t* empty) {
  asm volatile(
      "{\n\t.reg .pred p, q, e;\n\tsetp.ne.u32 p, %9, %9;\n\tsetp.eq.u32 q, %9, %9;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %5, %9, p;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %2, %6, %9, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %3, %7, %9, q;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %4, %8, %9, q;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%10];\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%11];\n\t}"
      ::"r"(d_tmem), "l"(a_desc), "l"(a_desc + 2), "l"(a_desc + 4), "l"(a_desc + 6), "l"(b_desc), "l"(b_desc + 2),
        "l"(b_desc + 4), "l"(b_desc + 6), "r"(idesc), "r"(smem_u32(done)), "r"(smem_u32(empty))
      : "memory");
}

// kN FP32 columns of this warp's 32 tensor-memory lanes, not waited for, and
// the wait for them: the registers pass through it so that no use of them
// moves above it.
template <int kN>
struct TmemLd;
template <>
struct TmemLd<8> {
  static __device__ __forceinline__ void start(uint32_t taddr, uint32_t (&r)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
        : "r"(taddr));
  }
  static __device__ __forceinline__ void wait(uint32_t (&r)[8]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7])
                 :
                 : "memory");
  }
};
template <>
struct TmemLd<16> {
  static __device__ __forceinline__ void start(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15])
        : "r"(taddr));
  }
  static __device__ __forceinline__ void wait(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                   "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
  }
};
template <>
struct TmemLd<32> {
  static __device__ __forceinline__ void start(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
          "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
          "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
  }
  static __device__ __forceinline__ void wait(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                   "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]),
                   "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]),
                   "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]),
                   "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :
                 : "memory");
  }
};

// Registers of the calling warpgroup's threads.
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Two FP32 values in one 64-bit register, and acc += a * b on them.
__device__ __forceinline__ uint64_t pack2(uint32_t lo, uint32_t hi) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "r"(lo), "r"(hi));
  return v;
}
__device__ __forceinline__ float pair_lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float pair_hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ void fma2(uint64_t& acc, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(acc) : "l"(a), "l"(b));
}

// Wait of a converged warp, polling at most `limit` times.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, uint32_t limit) {
#pragma unroll 1
  for (uint32_t i = 0; i < limit; ++i)
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return false;
}

__device__ __forceinline__ void cp_async_4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
// An arrival on `bar` once this thread's copies so far are complete.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// One finished output value (with the addend, if any).
__device__ __forceinline__ void f8_store_one(const Fp8Args& a, int m, int n, float v) {
  if (a.add) v += __bfloat162float(a.add[(int64_t)m * a.add_row + n]);
  const int64_t o = (int64_t)m * a.out_row + n;
  if (a.out_f32)
    static_cast<float*>(a.out)[o] = v;
  else
    static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ void st_32_bytes(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Eight consecutive columns of one output row.
__device__ __forceinline__ void f8_store_8(const Fp8Args& a, int m, int n, const float* v) {
  if (!a.vec || n + 8 > a.N) {
    for (int i = 0; i < 8; ++i)
      if (n + i < a.N) f8_store_one(a, m, n + i, v[i]);
    return;
  }
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = v[i];
  if (a.add) {
    const uint4 u = *reinterpret_cast<const uint4*>(a.add + (int64_t)m * a.add_row + n);
    const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[2 * i] += __uint_as_float(p[i] << 16);
      w[2 * i + 1] += __uint_as_float(p[i] & 0xffff0000u);
    }
  }
  if (a.out_f32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + (int64_t)m * a.out_row + n);
    o[0] = make_float4(w[0], w[1], w[2], w[3]);
    o[1] = make_float4(w[4], w[5], w[6], w[7]);
  } else {
    uint32_t p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(w[2 * i], w[2 * i + 1]);
      p[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + (int64_t)m * a.out_row + n) =
        make_uint4(p[0], p[1], p[2], p[3]);
  }
}

// kCols columns of the warp's 32 rows m0 .. (lane l holds row m0 + l) where
// rows allow no vector stores: sixteen at a time through shared memory (`part`,
// the warp's own), so that a store's lanes lie along a row.  One copy of the
// storing code, not one per sixteen columns: the loop is short, its
// instructions are fetched anew for every tile.
template <int kCols, int kOutRow>
__device__ __forceinline__ void f8_store_odd(const Fp8Args& a, int m0, int lane, int n0, const uint64_t (&acc)[kCols / 2],
                                             float* part) {
  const int each = a.pairs ? 2 : 1;                             // columns of a lane
  const int c = a.pairs ? 2 * (lane & 7) : lane & 15;           // of sixteen
  const int row0 = a.pairs ? lane >> 3 : lane >> 4, rows = 2 * each;
#pragma unroll 1
  for (int g = 0; g < kCols / 16; ++g) {
#pragma unroll
    for (int i = 0; i < kCols / 16; ++i)
      if (i == g) {
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          part[lane * kOutRow + 2 * p] = pair_lo(acc[8 * i + p]);
          part[lane * kOutRow + 2 * p + 1] = pair_hi(acc[8 * i + p]);
        }
      }
    __syncwarp();
    const int n = n0 + 16 * g + c;
    if (n < a.N) {
      const bool two = each == 2 && n + 1 < a.N;
      const int size = a.out_f32 ? 4 : 2;
      char* o = static_cast<char*>(a.out) + ((int64_t)(m0 + row0) * a.out_row + n) * size;
      const int64_t step = a.out_row * rows * size;
      const __nv_bfloat16* add = a.add ? a.add + (int64_t)(m0 + row0) * a.add_row + n : nullptr;
#pragma unroll 4
      for (int r = row0; r < 32; r += rows, o += step) {
        float lo = part[r * kOutRow + c], hi = part[r * kOutRow + c + each - 1];
        if (m0 + r < a.M) {
          if (add) {
            lo += __bfloat162float(add[0]);
            if (two) hi += __bfloat162float(add[1]);
            add += a.add_row * rows;
          }
          if (a.out_f32) {
            if (two)
              *reinterpret_cast<float2*>(o) = make_float2(lo, hi);
            else
              *reinterpret_cast<float*>(o) = lo;
          } else {
            if (two)
              *reinterpret_cast<__nv_bfloat162*>(o) = __floats2bfloat162_rn(lo, hi);
            else
              *reinterpret_cast<__nv_bfloat16*>(o) = __float2bfloat16_rn(lo);
          }
        }
      }
    }
    __syncwarp();
  }
}

// Sixteen consecutive columns of one output row, in 32-byte stores where the
// rows allow them: lanes hold rows of their own, and a store of less than a
// sector of each writes the sector twice.
__device__ __forceinline__ void f8_store_16(const Fp8Args& a, int m, int n, float* v) {
  if (a.vec < 2 || n + 16 > a.N) {
    if (n < a.N) f8_store_8(a, m, n, v);
    if (n + 8 < a.N) f8_store_8(a, m, n + 8, v + 8);
    return;
  }
  if (a.add) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 u = *reinterpret_cast<const uint4*>(a.add + (int64_t)m * a.add_row + n + 8 * h);
      const uint32_t p[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[8 * h + 2 * i] += __uint_as_float(p[i] << 16);
        v[8 * h + 2 * i + 1] += __uint_as_float(p[i] & 0xffff0000u);
      }
    }
  }
  uint32_t w[8];
  if (a.out_f32) {
    float* o = static_cast<float*>(a.out) + (int64_t)m * a.out_row + n;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * h + i]);
      st_32_bytes(o + 8 * h, w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    st_32_bytes(static_cast<__nv_bfloat16*>(a.out) + (int64_t)m * a.out_row + n, w);
  }
}

// Four consecutive columns of one output row.
__device__ __forceinline__ void f8_store_4(const Fp8Args& a, int m, int n, float4 v) {
  if (!a.vec || n + 4 > a.N) {
    const float w[4] = {v.x, v.y, v.z, v.w};
    for (int i = 0; i < 4; ++i)
      if (n + i < a.N) f8_store_one(a, m, n + i, w[i]);
    return;
  }
  if (a.add) {
    const uint2 u = *reinterpret_cast<const uint2*>(a.add + (int64_t)m * a.add_row + n);
    v.x += __uint_as_float(u.x << 16);
    v.y += __uint_as_float(u.x & 0xffff0000u);
    v.z += __uint_as_float(u.y << 16);
    v.w += __uint_as_float(u.y & 0xffff0000u);
  }
  if (a.out_f32) {
    *reinterpret_cast<float4*>(static_cast<float*>(a.out) + (int64_t)m * a.out_row + n) = v;
  } else {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + (int64_t)m * a.out_row + n) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Four floats at `saddr` (a shared-memory address of this CTA) in CTA `rank`
// of the cluster.
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t saddr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .u32 ra;\n\tmapa.shared::cluster.u32 ra, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [ra];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(saddr), "r"(rank)
      : "memory");
  return v;
}

// Persistent tile loop: CTA b computes tiles b, b + gridDim.x, ... of the
// m_tiles x n_tiles grid (token tiles fastest).  map_a: the 128-row
// operand's bytes, box 128 rows x 128 B; map_b: the other operand's, box BN
// rows x 128 B; both SWIZZLE_128B, zero-filled past their rows and past K.
//
// kSplit (a cluster of `split` CTAs per tile, one tile per
// cluster): the CTAs of a cluster take consecutive ranges of the K blocks,
// leave their partial tiles in their shared memory, and each sums the
// cluster's partials, in rank order, for its share of the tile's tokens and
// stores them.
//
// kXq > 0 (with kSplit; at most kXq K blocks per CTA): the scale warps and
// four more first quantise the BF16 tokens of the CTA's K range into shared memory,
// in the swizzled layout the MMA reads, while the weights are on their way.
// At most eight tokens: what the MMA's other rows read reaches only
// accumulator columns that are not stored.
template <int BN, bool kSwap, bool kTwo = false, bool kSplit = false, int kXq = 0>
__device__ __forceinline__ void gemm_fp8_persistent(const CUtensorMap* map_a, const CUtensorMap* map_b,
                                                    const Fp8Args& a, uint32_t* err, int split = 1) {
  using Cfg = F8Cfg<BN, kSwap, kTwo, kXq>;
  constexpr bool kFuse = Cfg::kFuse;
  static_assert(kSplit || !kSwap, "few tokens: one tile per cluster");
  static_assert(!kSplit || !Cfg::kMoveRegs, "every warp joins the cluster's sums");
  constexpr int S = Cfg::kStages, NA = Cfg::kAcc;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
  uint8_t* xq = smem + S * Cfg::kStageBytes;                                // [kXq][8][128]
  constexpr int kChunk = Cfg::kChunk, kChunks = Cfg::kChunks;
  float* xsc = reinterpret_cast<float*>(xq + Cfg::kXqBytes);                // [kChunks][kChunk][kXRows]
  float* wsc = xsc + kChunks * kChunk * Cfg::kXRows;                        // [kChunks][kChunk][kWBlocks]
  uint64_t* full = reinterpret_cast<uint64_t*>(wsc + kChunks * kChunk * Cfg::kWBlocks);
  uint64_t* empty = full + S;
  uint64_t* done = empty + S;     // [NA]
  uint64_t* accfree = done + NA;  // [NA]
  uint64_t* xready = accfree + NA;  // kXq: the tokens are quantised
  uint64_t* sfull = xready + 1;  // [kChunks] a chunk of scales has arrived
  uint64_t* sempty = sfull + kChunks;  // [kChunks] ... and was used
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sempty + kChunks);
  float* outs = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(full) + Cfg::kBarBytes);  // [kScaleWarps][32][kOutRow]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int m_tiles = (a.M + Cfg::kXRows - 1) / Cfg::kXRows;
  const int n_tiles = (a.N + Cfg::kWRows - 1) / Cfg::kWRows;
  const int tiles = m_tiles * n_tiles;
  const int nk_all = (a.K + kF8BK - 1) / kF8BK;
  // this CTA's K blocks and its first tile
  const int rank = kSplit ? (int)(blockIdx.x % split) : 0;
  const int kb0 = kSplit ? (int)((int64_t)nk_all * rank / split) : 0;
  const int nk = (kSplit ? (int)((int64_t)nk_all * (rank + 1) / split) : nk_all) - kb0;
  const int first = kSplit ? (int)(blockIdx.x / split) : (int)blockIdx.x;
  const int step = kSplit ? tiles : (int)gridDim.x;

  // the producer's loads of local K block s
  auto load_w = [&](int slot, int s, int w0) {
    uint8_t* st = smem + slot * Cfg::kStageBytes;
    mbar_arrive_expect_tx(&full[slot], Cfg::kStageBytes);
    tma_load_2d(kSwap ? st : st + Cfg::kStageA, kSwap ? map_a : map_b, (kb0 + s) * kF8BK, w0, &full[slot]);
  };
  auto load_x = [&](int slot, int s, int x0) {
    uint8_t* st = smem + slot * Cfg::kStageBytes;
    tma_load_2d(kSwap ? st + Cfg::kStageA : st, kSwap ? map_b : map_a, (kb0 + s) * kF8BK, x0, &full[slot]);
  };
  const int ahead = first < tiles ? (nk < S ? nk : S) : 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < NA; ++b) {
      mbar_init(&done[b], 1);
      mbar_init(&accfree[b], Cfg::kScaleWarps);
    }
    mbar_init(xready, Cfg::kScaleWarps + Cfg::kQuantWarps);
    for (int b = 0; b < kChunks; ++b) {
      mbar_init(&sfull[b], 32);
      mbar_init(&sempty[b], Cfg::kScaleWarps);
    }
    fence_mbar_init();
    // this thread is the producer: the first stages' weights set out at once
    if (!a.early) pdl_wait();
    for (int s = 0; s < ahead; ++s) load_w(s, s, (first / m_tiles) * Cfg::kWRows);
    if (!kFuse) tma_prefetch_desc(map_b);
  }
  // kXq: the scale and quantiser warps' half-warps take a K block of 128
  // values of a row each, lane l of 16 eight of them: half-warp h the local
  // K block h % 16 (h % 8 where a CTA has no more) of every row (every second
  // row).  The first rows set out here too.
  constexpr int kAhead = 4;
  const int qh = (int)(threadIdx.x - 32 * Cfg::kFirst) / 16, ql = lane & 15;
  const int qkb = nk > 8 ? qh & 15 : qh & 7, qr = nk > 8 ? qh >> 4 : qh >> 3;
  const int qstep = 2 * (Cfg::kScaleWarps + Cfg::kQuantWarps) / (nk > 8 ? 16 : 8);
  const int qk = (kb0 + qkb) * kF8BK + ql * 8;
  const int used = a.M < Cfg::kXRows ? a.M : Cfg::kXRows;  // (kXq: one token tile)
  uint4 raw[kFuse ? kAhead : 1];
  auto load_rows = [&](int r0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int r = r0 + i * qstep;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (qkb < nk && r < used && qk < a.K)
        raw[i] = *reinterpret_cast<const uint4*>(a.xb + (int64_t)r * a.xb_row + qk);
    }
  };
  if constexpr (kFuse) {
    if (warp >= Cfg::kFirst) {
      pdl_wait();
      load_rows(qr);
    }
  }
  // (This CTA may be resident before the launch before it is complete, and the
  // allocation waits until the columns are free.  It never holds columns that
  // a CTA of that launch still needs: CTAs of this library that fit beside a
  // kTwo CTA in shared memory, its own kind and the decode band's, take at
  // most 256 columns, and beside the others none fits.)
  if (warp == 1) tmem_alloc(tmem_slot, Cfg::kTmemCols);
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  auto quantise = [&]() {
    for (int r0 = qr; r0 < used; r0 += kAhead * qstep) {  // (the same rows for a whole warp)
      if (r0 != qr) load_rows(r0);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int r = r0 + i * qstep;
        float v[8];
        bf16x8_to_float(raw[i], v);
        const float sc = block_scale(block_amax(v));
        if (qkb < nk && r < used) {
          *reinterpret_cast<uint2*>(xq + qkb * 1024 + r * kF8BK + (((ql >> 1) ^ (r & 7)) << 4) + (ql & 1) * 8) =
              e4m3_quotients(v, sc);
          if (ql == 0) xsc[qkb * BN + r] = sc;
        }
      }
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(xready);
  };
  // (the registers move: 384 threads x 168 at launch = 128 x 104 + 256 x 200)
  if (warp < Cfg::kFirst) {
    if (Cfg::kMoveRegs) regs_dec<104>();
    if (warp == 0) {
      if (lane == 0) {
        pdl_wait();
        int g = 0;
        bool ok = true;
        for (int idx = first; ok && idx < tiles; idx += step) {
          const int x0 = (idx % m_tiles) * Cfg::kXRows, w0 = (idx / m_tiles) * Cfg::kWRows;
          for (int s = 0; s < nk; ++s, ++g) {
            const int slot = g % S, round = g / S;
            if (round > 0 && !mbar_wait(&empty[slot], (round - 1) & 1, err, 1u)) {
              ok = false;
              break;
            }
            if (g >= ahead) load_w(slot, s, w0);
            if (!kFuse) load_x(slot, s, x0);
          }
        }
        if (!ok)  // gave up: see the copies under way in before the CTA ends
          for (int q = g > S ? g - S : 0; q < g; ++q) mbar_wait(&full[q % S], (q / S) & 1, err, 16u);
      }
    } else if (warp <= Cfg::kMmaWarps) {
      constexpr uint32_t idesc = idesc_e4m3(kF8BM, BN);
      int g = 0;
      bool ok = !kFuse || __all_sync(0xffffffffu, mbar_wait(xready, 0, err, 8u));
      for (int idx = first; ok && idx < tiles; idx += step) {
        for (int s = 0; s < nk; ++s, ++g) {
          const int slot = g % S, round = g / S, ab = g % NA, use = g / NA;
          if (Cfg::kMmaWarps > 1 && ab % Cfg::kMmaWarps != warp - 1) continue;
          bool w = mbar_wait(&full[slot], round & 1, err, 2u);
          w = w && (use == 0 || mbar_wait(&accfree[ab], (use - 1) & 1, err, 2u));
          if (!__all_sync(0xffffffffu, w)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t acc = tmem + (uint32_t)(ab * BN);
          const uint64_t da = smem_desc(smem_u32(smem + slot * Cfg::kStageBytes), 16, 1024, kLayoutSW128);
          const uint8_t* bst = kFuse ? xq + s * 1024 : smem + slot * Cfg::kStageBytes + Cfg::kStageA;
          const uint64_t db = smem_desc(smem_u32(bst), 16, 1024, kLayoutSW128);
          mma_f8_block(acc, da, db, idesc, &done[ab], &empty[slot]);
        }
      }
    } else {
      // the scales of this CTA's K blocks [c0, c0 + kChunk) of every tile
      pdl_wait();
      int gc = 0;
      bool ok = true;
      for (int idx = first; ok && idx < tiles; idx += step) {
        const int x0 = (idx % m_tiles) * Cfg::kXRows, wb = (idx / m_tiles) * Cfg::kWRows / 128;
        const int last = (a.N - 1) / 128;
        for (int c0 = 0; c0 < nk; c0 += kChunk, ++gc) {
          const int buf = gc % kChunks, round = gc / kChunks;
          if (round > 0 && !warp_wait(&sempty[buf], (round - 1) & 1, kWaitPollLimit)) {
            if (lane == 0) atomicOr(err, 32u);
            ok = false;
            break;
          }
          const int n = nk - c0 < kChunk ? nk - c0 : kChunk;
          float* xd = xsc + buf * kChunk * Cfg::kXRows;
          if (!kFuse && !kSwap && a.xs_vec) {  // four rows a lane
            const int m = x0 + 4 * lane < a.M ? x0 + 4 * lane : 0;
            const float* from = a.xs + m + (int64_t)(kb0 + c0) * a.xs_blk;
            for (int k = 0; k < n; ++k, from += a.xs_blk) cp_async_16(xd + k * Cfg::kXRows + 4 * lane, from);
          } else if (!kFuse) {
            // (rows past M read the last row's scale; their sums are not stored)
#pragma unroll
            for (int r = lane; r < Cfg::kXRows; r += 32) {
              const int m = x0 + r < a.M ? x0 + r : a.M - 1;
              const float* from = a.xs + (int64_t)m * a.xs_row + (int64_t)(kb0 + c0) * a.xs_blk;
              for (int k = 0; k < n; ++k, from += a.xs_blk) cp_async_4(xd + k * Cfg::kXRows + r, from);
            }
          }
          float* wd = wsc + buf * kChunk * Cfg::kWBlocks;
          if (lane < n * Cfg::kWBlocks) {
            const int b = wb + lane % Cfg::kWBlocks;
            cp_async_4(wd + lane, a.ws + (int64_t)(b < last ? b : last) * a.ws_row + kb0 + c0 + lane / Cfg::kWBlocks);
          }
          cp_async_arrive(&sfull[buf]);
        }
      }
      cp_async_wait_all();
    }
  } else if (kFuse && warp >= Cfg::kFirst + Cfg::kScaleWarps) {
    if constexpr (kFuse) quantise();
  } else {
    if (Cfg::kMoveRegs) regs_inc<200>();
    const int half = (warp - Cfg::kFirst) / 4;
    const int row = (warp & 3) * 32 + lane;  // row of the 128-row operand (tensor-memory lane)
    const uint32_t tm = tmem + ((uint32_t)((warp & 3) * 32) << 16) + (uint32_t)(half * Cfg::kCols);
    pdl_wait();
    pdl_launch_dependents();
    int g = 0, gc = 0;
    uint32_t polls = kWaitPollLimit;  // 1 once a wait gave up: the warp then goes through its barriers without waiting
    if constexpr (kFuse) {
      quantise();
      // (the scales of the quantiser warps' rows)
      if (!warp_wait(xready, 0, polls)) {
        polls = 1;
        atomicOr(err, 8u);
      }
    }
    for (int idx = first; idx < tiles; idx += step) {
      const int x0 = (idx % m_tiles) * Cfg::kXRows, w0 = (idx / m_tiles) * Cfg::kWRows;
      uint64_t acc[Cfg::kCols / 2];  // pairs of sums
#pragma unroll
      for (int i = 0; i < Cfg::kCols / 2; ++i) acc[i] = 0;
      for (int c0 = 0; c0 < nk; c0 += kChunk, ++gc) {
        const int buf = gc % kChunks;
        if (!warp_wait(&sfull[buf], (gc / kChunks) & 1, polls)) {
          polls = 1;
          atomicOr(err, 32u);
        }
        const float* xd = xsc + buf * kChunk * Cfg::kXRows;
        const float* wd = wsc + buf * kChunk * Cfg::kWBlocks;
        const int n = nk - c0 < kChunk ? nk - c0 : kChunk;
        // The accumulator's columns pass through two register buffers.  A
        // wait for tensor-memory loads is for all of them, so both buffers'
        // loads fly together, each started as its buffer is used up.  (No
        // conditions here: with loads under a branch the compiler copies the
        // buffers.)
        constexpr int kLoads = Cfg::kCols / Cfg::kLd;
#pragma unroll 1
        for (int kk = 0; kk < n; ++kk, ++g) {
          const int ab = g % NA;
          const uint32_t src = tm + (uint32_t)(ab * BN);
          const float ws = wd[kk * Cfg::kWBlocks + (kSwap ? 0 : half * Cfg::kCols / 128)];
          const float rs = kSwap ? 0.f : xd[kk * Cfg::kXRows + row] * ws;
          const uint64_t rs2 = pack2(__float_as_uint(rs), __float_as_uint(rs));
          // acc += scales * (columns of load j)
          auto add = [&](int j, const uint32_t (&r)[Cfg::kLd]) {
#pragma unroll
            for (int i = 0; i < Cfg::kLd / 4; ++i) {
              uint64_t s0 = rs2, s1 = rs2;
              if (kSwap) {  // a scale per column, four at a time
                const float4 f =
                    *reinterpret_cast<const float4*>(xd + kk * Cfg::kXRows + half * Cfg::kCols + Cfg::kLd * j + 4 * i);
                s0 = pack2(__float_as_uint(f.x * ws), __float_as_uint(f.y * ws));
                s1 = pack2(__float_as_uint(f.z * ws), __float_as_uint(f.w * ws));
              }
              fma2(acc[Cfg::kLd / 2 * j + 2 * i], pack2(r[4 * i], r[4 * i + 1]), s0);
              fma2(acc[Cfg::kLd / 2 * j + 2 * i + 1], pack2(r[4 * i + 2], r[4 * i + 3]), s1);
            }
          };
          if (!warp_wait(&done[ab], (g / NA) & 1, polls)) {
            polls = 1;
            atomicOr(err, 4u);
          }
          tc_fence_after();
          uint32_t r0[Cfg::kLd], r1[Cfg::kLd];
          TmemLd<Cfg::kLd>::start(src, r0);
          TmemLd<Cfg::kLd>::start(src + Cfg::kLd, r1);
#pragma unroll
          for (int j = 0; j < kLoads; j += 2) {
            TmemLd<Cfg::kLd>::wait(r0);
            TmemLd<Cfg::kLd>::wait(r1);
            if (j + 2 == kLoads) {  // the accumulator is read out
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&accfree[ab]);
            }
            add(j, r0);
            if (j + 2 < kLoads) TmemLd<Cfg::kLd>::start(src + Cfg::kLd * (j + 2), r0);
            add(j + 1, r1);
            if (j + 2 < kLoads) TmemLd<Cfg::kLd>::start(src + Cfg::kLd * (j + 3), r1);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sempty[buf]);
      }
      if (kSplit) {
        // the ring is idle: every load was multiplied, every MMA is done
        float* part = reinterpret_cast<float*>(smem);
        if (kSwap) {
#pragma unroll
          for (int i = 0; i < Cfg::kCols / 2; ++i) {
            const int c = half * Cfg::kCols + 2 * i;
            part[c * Cfg::kPartRow + row] = pair_lo(acc[i]);
            part[(c + 1) * Cfg::kPartRow + row] = pair_hi(acc[i]);
          }
        } else {
          float4* p = reinterpret_cast<float4*>(part + row * Cfg::kPartRow + half * Cfg::kCols);
#pragma unroll
          for (int i = 0; i < Cfg::kCols / 4; ++i)
            p[i] = make_float4(pair_lo(acc[2 * i]), pair_hi(acc[2 * i]), pair_lo(acc[2 * i + 1]), pair_hi(acc[2 * i + 1]));
        }
        continue;
      }
      if (polls == 1) continue;
      if constexpr (!kSwap) {
        __syncwarp();
        const int m0 = x0 + (warp & 3) * 32;
        const int n0 = w0 + half * Cfg::kCols;
        if (a.vec == 0) {
          f8_store_odd<Cfg::kCols, Cfg::kOutRow>(a, m0, lane, n0, acc, outs + (warp - Cfg::kFirst) * 32 * Cfg::kOutRow);
        } else if (m0 + lane < a.M) {
#pragma unroll
          for (int i = 0; i < Cfg::kCols / 16; ++i) {
            float v[16];
#pragma unroll
            for (int p = 0; p < 8; ++p) v[2 * p] = pair_lo(acc[8 * i + p]), v[2 * p + 1] = pair_hi(acc[8 * i + p]);
            if (n0 + 16 * i < a.N) f8_store_16(a, m0 + lane, n0 + 16 * i, v);
          }
        }
      }
    }
  }
  if (kSplit) {
    __syncwarp();
    cluster_sync();
    const int x0 = (first % m_tiles) * Cfg::kXRows, w0 = (first / m_tiles) * Cfg::kWRows;
    const int used = a.M - x0 < Cfg::kXRows ? a.M - x0 : Cfg::kXRows;  // tokens of this tile
    const int c0 = used * rank / split, c1 = used * (rank + 1) / split;
    constexpr int kQuads = Cfg::kWRows / 4;
    for (int e = threadIdx.x; e < (c1 - c0) * kQuads; e += Cfg::kThreads) {
      const int c = c0 + e / kQuads, r = e % kQuads * 4;
      const uint32_t at = smem_u32(smem) + (uint32_t)(c * Cfg::kPartRow + r) * 4;
      float4 v = ld_cluster_f4(at, 0);
      for (int p = 1; p < split; ++p) {
        const float4 u = ld_cluster_f4(at, (uint32_t)p);
        v.x += u.x;
        v.y += u.y;
        v.z += u.z;
        v.w += u.w;
      }
      if (w0 + r < a.N) f8_store_4(a, x0 + c, w0 + r, v);
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while another reads its partials
  }
  tc_fence_before();
  __syncwarp();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, Cfg::kTmemCols);
}

}  // namespace moe_fp4
