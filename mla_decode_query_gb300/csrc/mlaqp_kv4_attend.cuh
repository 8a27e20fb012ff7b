// MLA decode attention over the paged 4-bit latent cache on the tcgen05
// tensor cores of sm_103a.
//
// Mathematics.  A cached token t has E2M1 codes c with block scales
// 2^(s_j-127).  With s_t the largest of its 16 scale bytes,
//   latent[t,n] = K8[t,n] * 2^(s_t-133),   K8 = code * 2^(s_j-s_t+6)
// and K8 is exact in E4M3 while s_t - s_j <= 14 (below that it rounds, at
// 2^-16 of the token's largest step).  So one 8-bit tile K8 [tokens][512]
// serves both products:
//   scores  D[t,r]  = sum_n K8[t,n] * Q8[r,n]         A = K8, rows = tokens
//   output  O[n,r] += sum_t K8[t,n] * P8[t,r]         A = K8 transposed
// with the 16 or 32 query rows r = (query token, head) on the narrow N side
// of the MMA (swap-AB), and the token's scale folded into a number per (t,r)
// in registers:
//   y = (D * 2^(s_t-133) + Dr) * C_r + (s_t-133)      log2 units
//   P = 2^(y - M_r + 12)     l_r += P * 2^(133-s_t)   M_r the running maximum
//   x[r,n] = O[n,r] / l_r    lse_r = ln l_r + (M_r-12) ln 2
//   (l_r = 0, no token there to be seen: 0 and -infinity)
// Dr is the rope part, a BF16 product of its own; C_r holds the softmax
// scale, log2 e and the row's power of two.
//
// 8-bit operands without loss of the inputs' precision:
//   Q   BF16 rows are scaled to a maximum in [128,256) and split into two
//       E4M3 terms hi + lo/16: a BF16 significand has 8 bits, two terms of 4
//       hold it down to E4M3's smallest normal in hi, 2^-13 of the maximum or
//       less; below, steps of lo's smallest subnormal remain, 2^-20 of the
//       maximum (a third term would want 8 KB of shared memory that is not
//       there).  E4M3 queries are used as they are.  The terms are extra N rows.
//   P   FP16 (11 bits) as three E5M2 terms, each rounded to nearest, again
//       extra N rows: together exactly that FP16 number down to 2^-18 of the
//       maximum (of p_t * 2^s_t over the tokens), and absolute steps of 2^-28
//       below, so that 2^17 tokens far below the maximum still add up.  l sums
//       the FP32 values: statistics keep 32 bits.
// The MMAs cost what the A tile's reads from shared memory cost, so the
// extra rows are free.
//
// Work split.  The sequences' 128-token tiles form one line; CTA c of the
// grid (one per SM) takes an equal stretch of it, whatever the lengths.  A
// stretch that holds a whole sequence writes x; the others leave (O, M, l)
// in the workspace and the join kernel adds the pieces in order.  (One CTA
// per sequence would leave SMs idle for few sequences or mixed lengths; a
// split of each sequence into a fixed number of pieces does for long ones.)
//
// A CTA is a pipeline of warps:
//   warp 16      copies pages into shared memory (bulk copies: codes and
//                scales in units of 64 tokens, rope rows straight into the
//                swizzled tile, the cache's layout being that of the tile);
//   warp 19      scale bytes -> s_t and s_t - s_j, a token per lane;
//   warps 8-15   codes -> E4M3: a byte permute looks four magnitudes up in
//                the eight values of their block's scale;
//   warps 17, 18 issue the MMAs of scores and output;
//   warps 0-7    queries, softmax (one token and half of the rows per
//                thread), rescaling, output.
// O stays in tensor memory; it is rescaled only when a row's maximum has
// grown by more than 2^3.
//
// What bounds it (GB300, 152 SMs, H = 16).  64 sequences of 16000 to 32768
// tokens, E4M3 queries: 149 us, 4.29 TB/s of cache and rows, 63% of the copy
// rate of 6.79 TB/s.  A tile takes an SM 3000 to 3300 cycles; its bytes alone
// would take 2230, its 36 MMAs 2155 (some 60 each whatever N is).  What is
// left is the way of a tile through the pipeline: scores 2500 cycles beside
// the output product before, softmax 2100, output 2000, conversion of the
// tile that takes its place 1300, over two K8 tiles; a third one (64 KB) does
// not fit.  Short calls (32 sequences of up to 8191 tokens: 27.2 us, 2.1 TB/s;
// one of 131071: 24.7 us, 2.1 TB/s; six or seven tiles per SM) spend 15000
// cycles, 8 us, until the first probabilities, and 5 to 6 us in the join.
#pragma once

#include "mlaqp_kernel_large.cuh"
#include "mlaqp_kv4.cuh"
#include "mlaqp_kv4_launch.h"

namespace mlaqp {

constexpr int kAttThreads = 640;
constexpr int kAttRegs = 96;    // a thread's at launch: 65536 / 640 in steps of 8
constexpr int kAttSoftWarps = 8;   // two groups of four, each with half of the rows
constexpr int kAttDequantWarps = 8;
constexpr int kAttLoadWarp = kAttSoftWarps + kAttDequantWarps;
constexpr int kAttScoreWarp = kAttLoadWarp + 1;
constexpr int kAttOutputWarp = kAttLoadWarp + 2;
constexpr int kAttScaleWarp = kAttLoadWarp + 3;
constexpr int kAttTile = 128;   // tokens per tile (MMA M of the scores)
// Tiles whose scales are kept.  While the softmax still reads those of tile
// k-2, the code warps may have fetched tile k+1 and the scale warp be three
// copy units, a tile and a half, ahead of them: k-2 .. k+3.
constexpr int kAttScaleTiles = 6;
constexpr int kAttPageTiles = 4;   // tiles whose rope rows may be outstanding
constexpr int kAttMaskTiles = 8;   // the same for what the copying warp notes, which is ahead of both
constexpr int kAttMaxSeqs = 256;  // sequences x row groups of a call
constexpr float kAttSlack = 3.f;  // log2 growth of the maximum that is let pass
constexpr float kAttShift = 12.f; // 2^(12+3) stays inside E5M2 and FP16

// A row group's tiles are followed by so many places on the line without a
// tile: what its end costs a CTA (sums, output, the pipeline empty), in tiles.
// 32 sequences of up to 8191 tokens: 34.1 us with none, 30.1, 28.9, 29.2 and
// 29.0 with one to four; 16 of up to 4100, 4 query tokens: 32.8, 30.4, 30.0,
// 30.6, 30.7.
constexpr int kAttEndTiles = 2;

// Reference of a row that has seen no token: whatever it sees first is above.
constexpr float kAttUnseen = -1e30f;

constexpr int kRopeTile = kAttTile * kKv4RopeBytes;
constexpr int kK8Block = kAttTile * 128;  // 128 latents of a tile
constexpr int kK8Tile = 4 * kK8Block;

// What follows from the lengths, and the limit of the waits.
struct AttSchedule {
  int prefix[kAttMaxSeqs + 1];  // length of the line before each row group
  int len[kAttMaxSeqs];
  int scan[8];
  int cut, begin, end, group;  // this CTA's stretch, its first tile, that tile's row group
  uint32_t wait_ns;  // 0: a wait ran out
  int units, ropes;  // copy units and rope tiles asked for, when the copying warp has ended
};

template <int R, int Ring>  // Ring: tokens of all copy units in flight
struct AttShared : AttSchedule {
  uint32_t tmem;
  alignas(8) uint32_t lut[32][2];           // E4M3 of the 8 magnitudes * 2^(6-k)
  alignas(16) uint8_t rel[Ring * kKv4Blocks];  // s_t - s_j of the copy units, at most 31
  // by warp, for its half of the rows
  alignas(16) float wmax[kAttSoftWarps][R / 2];
  alignas(16) float mref[kAttSoftWarps][R / 2];  // M_r - 12, or kAttUnseen
  alignas(16) float alpha[kAttSoftWarps][R / 2];
  // of the row group at hand and the next one, by turns
  alignas(16) float cr[2][R];               // C_r
  int limit[2][R];                          // visible tokens of a row
  alignas(8) int64_t xoff[2][R];            // its place in x, -1: padding
  int lseoff[2][R];
  uint8_t smax[kAttScaleTiles][kAttTile];   // s_t
  uint32_t tmask[kAttMaskTiles];            // 16-token parts of a tile that were copied, a bit each
  int pages[kAttPageTiles][8];              // a tile's pages, -1: none
  alignas(8) uint64_t bars[42];
};

// Shared memory and tensor memory of a variant: R query rows, E4M3 or BF16
// queries.  Units copy units of Unit tokens take what the K8 tiles, queries
// and P leave: 64 tokens a unit where two of them fit, because a warp that
// works alone needs some hundred cycles a unit whatever its size.
template <int R, bool E4>
struct AttPlan {
  static constexpr int QTerms = E4 ? 1 : 2;
  static constexpr int NQ = QTerms * R;            // N of the score MMA
  static constexpr int NP = 3 * R;                 // N of the output MMA
  static constexpr int SCols = NQ + R;             // scores + rope part
  static constexpr int SBufs = (R == 32 && !E4) ? 1 : 2;
  static constexpr int OCol = SBufs * SCols;
  static constexpr int Unit = (R == 32 && !E4) ? 32 : 64;
  static constexpr int Units = (R == 32 && E4) ? 2 : 3;
  static constexpr int RopeBufs = 1;
  static constexpr int PerTile = kAttTile / Unit;
  static_assert(Units <= 2 * PerTile, "the scale barriers are the units of two tiles, waited for once each");
  static constexpr int WarpTokens = kAttTile / (kAttDequantWarps / 4);  // tokens of a code warp
  static constexpr int UnitWarps = 4 * (Unit > WarpTokens ? Unit / WarpTokens : 1);  // code warps that read a unit
  static constexpr int HalfRows = R / 2;                         // rows of a softmax warp

  static constexpr int UnitCodes = Unit * kKv4CodeBytes;
  static constexpr int UnitBytes = UnitCodes + Unit * kKv4Blocks;
  using Shared = AttShared<R, Unit * Units>;
  static constexpr int K8 = 0;
  static constexpr int Rope = K8 + 2 * kK8Tile;
  static constexpr int Q = Rope + RopeBufs * kRopeTile;
  static constexpr int QBlock = NQ * 128;          // 128 latents of the queries
  static constexpr int QPe = Q + 4 * QBlock;
  static constexpr int P = QPe + R * 128;
  static constexpr int PChunk = 16 * kAttTile;     // 16 rows of P
  static constexpr int Raw = P + NP / 16 * PChunk;
  static constexpr int Misc = Raw + Units * UnitBytes;
  static constexpr int Bytes = Misc + static_cast<int>(sizeof(Shared));
  static_assert(OCol + 4 * NP <= 512, "tensor memory");
  static_assert(Bytes <= 232448, "shared memory");
  // registers of the softmax, code and other warps, of the five warpgroups' at launch
  static constexpr int SoftRegs = R == 16 ? 96 : 112, CodeRegs = R == 16 ? 96 : 88, OtherRegs = R == 16 ? 96 : 80;
  static_assert(2 * SoftRegs + kAttDequantWarps / 4 * CodeRegs + OtherRegs <= 5 * kAttRegs, "registers");
  // barrier indexes; K8Full and K8Empty: 4 * tile buffer + block of 128 latents
  static constexpr int RawFull = 0, RawEmpty = RawFull + Units, ScaleFull = RawEmpty + Units,
                       RopeFull = ScaleFull + 2 * PerTile,
                       RopeEmpty = RopeFull + RopeBufs, K8Full = RopeEmpty + RopeBufs, K8Empty = K8Full + 8,  // per 128 latents of a tile
                       SFull = K8Empty + 8, SEmpty = SFull + SBufs, PFull = SEmpty + SBufs, PvDone = PFull + 1,
                       QFull = PvDone + 1, OEmpty = QFull + 1, Drain = OEmpty + 1, BarCount = Drain + 2;
  static_assert(BarCount <= 42, "barriers");
  static_assert(Drain - OEmpty == 1 && QFull - PvDone == 1, "kAttStages hand-overs, in this order");
};

// Instruction descriptor: FP32 accumulator, operand formats and majors.
__host__ __device__ constexpr uint32_t att_idesc(int m, int n, int afmt, int bfmt, bool a_mn, bool b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(afmt) << 7) | (static_cast<uint32_t>(bfmt) << 10) |
         (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}
constexpr int kFmtE4M3 = 0, kFmtE5M2 = 1, kFmtBf16 = 1;

// Descriptor of an unswizzled operand (bits 61..63 = 0).
__device__ __forceinline__ uint64_t smem_desc_plain(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  uint64_t d = static_cast<uint64_t>((addr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;
  d |= static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  return d;
}

__device__ __forceinline__ void umma_f8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// N (8 or 16) columns of this thread's TMEM lane: begun, not there before
// tmem_ld_end(), which makes the registers depend on the wait.
#define MLAQP_R8(c, r, o) \
  c(r[o]), c(r[o + 1]), c(r[o + 2]), c(r[o + 3]), c(r[o + 4]), c(r[o + 5]), c(r[o + 6]), c(r[o + 7])
template <int N>
__device__ __forceinline__ void tmem_ld_begin(uint32_t a, uint32_t* r) {
  static_assert(N == 8 || N == 16, "columns");
  if constexpr (N == 8)
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : MLAQP_R8("=r", r, 0)
                 : "r"(a)
                 : "memory");
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : MLAQP_R8("=r", r, 0), MLAQP_R8("=r", r, 8)
        : "r"(a)
        : "memory");
}
template <int N>
__device__ __forceinline__ void tmem_ld_end(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t a, const uint32_t (&r)[N]) {
  static_assert(N == 8 || N == 16, "columns");
  if constexpr (N == 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::MLAQP_R8("r", r, 0), "r"(a)
                 : "memory");
  else
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::MLAQP_R8("r", r, 0),
        MLAQP_R8("r", r, 8), "r"(a)
        : "memory");
}
#undef MLAQP_R8
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A warpgroup's registers a thread from here on (kAttRegs before).
template <int N>
__device__ __forceinline__ void att_set_regs() {
  static_assert(N % 8 == 0 && N >= 24 && N <= 256, "registers");
  if constexpr (N > kAttRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  if constexpr (N < kAttRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// True for one lane of the (whole) warp, always the same.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}

// Whether the phase of that parity has completed; does not wait.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
  uint32_t d;
  asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
  return d;
}

// Barrier of a group of four softmax warps (group 0 or 1); the second form
// tells whether any thread says yes.  Every one of these warps passes every
// barrier, also when it has given up.
__device__ __forceinline__ void soft_barrier(int group) {
  asm volatile("barrier.sync %0, 128;" ::"r"(1 + group) : "memory");
}
__device__ __forceinline__ bool soft_barrier_any(int group, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "barrier.red.or.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(1 + group), "r"(static_cast<uint32_t>(mine))
      : "memory");
  return any != 0;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Largest value of the warp; NaNs are left out.
__device__ __forceinline__ float warp_max(float v) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Everything that follows from the lengths: the tiles of each row group and
// the stretch of this CTA.  All threads call.
__device__ __forceinline__ int att_schedule(const Kv4AttendParams& p, int R, AttSchedule& s, bool tell) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = (p.q_len * p.H + R - 1) / R;
  const int V = p.B * groups;
  int tiles = 0;
  if (tid < kAttMaxSeqs) {
    int len = 0;
    if (tid < V) {
      const int b = tid / groups, g = tid % groups;
      const int seq = p.seqs ? p.seqs[b] : b;
      bool bad = seq < 0 || seq >= p.num_seqs;
      if (!bad) {
        len = p.seq_lens[seq];
        // a sequence holds a page once, so the pool bounds its length too
        bad = len < 0 || len > p.table_stride << p.cache.shift || len > p.cache.num_pages << p.cache.shift;
      }
      if (bad) {
        if (tell) atomicOr(&g_device_status, kDevStatusBadIndex);
        len = 0;
      }
      // the group's last row sees the most
      const int last = min(g * R + R, p.q_len * p.H) - 1;
      const int seen = max(0, len - (p.q_len - 1 - last / p.H));
      tiles = static_cast<int>((static_cast<int64_t>(seen) + kAttTile - 1) / kAttTile);
      if (tiles > 0) tiles += kAttEndTiles;
    }
    s.len[tid] = len;
    int inc = tiles;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += u;
    }
    if (lane == 31) s.scan[warp] = inc;
    tiles = inc;
  }
  __syncthreads();
  if (tid < kAttMaxSeqs) {
    int before = 0;
    for (int w = 0; w < warp; ++w) before += s.scan[w];
    s.prefix[tid + 1] = before + tiles;
    if (tid == 0) s.prefix[0] = 0;
  }
  __syncthreads();
  return V;
}

// The line of `total` tiles cut into `n` stretches, one or more tiles each:
// stretch c begins at floor(total * c / n), kept in 32 bits by the quotient
// and remainder of total / n (n <= 256).
struct AttCut {
  int n, base, rem;
  __device__ __forceinline__ AttCut(int total, int ctas) {
    n = max(min(total, ctas), 1);
    base = total / n;
    rem = total - base * n;
  }
  __device__ __forceinline__ int begin(int c) const { return base * c + rem * c / n; }
  // The stretch that holds place t: the last c with total * c / n < t + 1.
  __device__ __forceinline__ int owner(int total, int t) const {
    return static_cast<int>((static_cast<uint64_t>(t + 1) * n - 1) / static_cast<uint32_t>(total));
  }
};
constexpr int kAttMaxCtas = 256;

// Workspace: for each row group, what the join kernel has to know of it; then
// the pieces, slot 2c for the one that begins CTA c's stretch, 2c+1 for one
// that begins inside it: R rows of 512 sums, then M and l of each row.
struct alignas(8) AttGroup {
  int slot;    // of its first piece; the others are slots 2c of the CTAs that follow
  int pieces;  // 0: no tile, 1: written by its CTA
};
constexpr int kAttGroupBytes = kAttMaxSeqs * static_cast<int>(sizeof(AttGroup));
template <int R>
__host__ __device__ constexpr int64_t att_slot_floats() { return R * (kLatent + 2); }

}  // namespace mlaqp
