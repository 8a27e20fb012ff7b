// Choosing the pages that a query token attends to: scores from the pages'
// digests, and the best of them.
//
// Score of page p for query token m, H heads: the bound
//   sum_h sum_c max over the page's tokens of q[h,c] * v[t,c]
//     <= sum_c up[c] * largest[c] + down[c] * smallest[c]
//   up[c] = sum_h max(q[h,c], 0)   down[c] = sum_h min(q[h,c], 0)
// which is linear in the digest: the heads are summed once per query token,
// and a page costs 1152 products whatever H is.  q is held in 12 bits (one
// power of two a token), so up and down fit 16 bits, the digest's numbers are 8:
// a dp2a is two products, and the sums stay below 2^31 (512 * 16 * 2047 * 127),
// exact, so the choice does not depend on the order of anything.
//
// Score kernel: the pages that have to be scored form one line over the
// sequences, and every CTA takes an equal stretch.  A warp takes four pages at a
// time, a lane 16 + 16 + 4 bytes of each digest; up and down lie in shared
// memory in the lanes' order, read once for four pages.  Bound by memory (1168
// bytes a page); the chain lengths -> queries -> up, down -> digests is what
// short calls wait for.
//
// Choice kernel: a CTA a query token.  The k-th highest score by histograms of
// 2048 places over the range that is still open (mostly two), then the pages
// from there on in order of position.

#include "mlaqp_dispatch.h"
#include "mlaqp_kv4.cuh"
#include "mlaqp_kv4_launch.h"
#include "mlaqp_kv4_step.h"

namespace mlaqp {

namespace {

constexpr int kSelectChunks = kOutDim / 8;           // of eight channels
constexpr int kSelectHeadGroups = 4;                 // heads h, h + 4, .. of a thread
constexpr int kSelectThreads = kSelectChunks * kSelectHeadGroups;
constexpr int kSelectWarps = kSelectThreads / 32;
constexpr int kSelectCtasPerSm = 2;
constexpr int kSelectMaxCluster = 8;
constexpr int kScorePages = 4;                       // in flight per warp
constexpr int kScoreWords = 18;                      // pairs of up / down of a lane: 8 + 8 + 2
constexpr int kScoreLane = 20;                       // a lane's words apart: 16-byte loads without bank conflicts
constexpr int kQueryWords = 32 * kScoreLane;         // of a query token
constexpr int kBatchBytes = kScorePages * 2 * kOutDim;  // of digests, without their exponents
constexpr int kStages = 2;                           // batches of a warp in shared memory
constexpr int kBins = 2048, kBinsLog = 11;
constexpr int kBinThreads = 256, kBinsEach = kBins / kBinThreads;
constexpr int kCandidates = 32;                      // keys that a warp ranks
constexpr int kHeldKeys = 2048;                      // keys and pages that stay in shared memory
constexpr int kChooseEach = 4;                       // pages of a thread in one sweep in order
static_assert(kSelectThreads % 32 == 0 && kSelectThreads >= kBinThreads, "whole warps, a thread for some bins");

// Dynamic shared memory: this, the warps' stages (later the bins), the queries' words.
struct SelectShared {
  uint32_t amax[kSelectWarps];
  uint32_t lo[kSelectWarps], hi[kSelectWarps];
  int scan[kSelectWarps][2];
  uint32_t from;   // first key of the place that holds the last one taken
  int above, in;   // keys above that place, in it
  int found;       // candidates
  uint32_t candidate[kCandidates];
  alignas(16) uint32_t keys[kHeldKeys];  // of this CTA's query tokens, one after the other
  union {
    alignas(16) uint32_t part[kSelectHeadGroups][kOutDim];  // up << 16 | -down, sums over a thread's heads
    alignas(16) int32_t pages[kHeldKeys];                   // (later) of the sequence, up to the last ones
  };
};
constexpr int kStagesAt = (sizeof(SelectShared) + 127) / 128 * 128;
constexpr int kWordsAt = kStagesAt + kSelectWarps * kStages * kBatchBytes;
static_assert(kBins * 4 <= kSelectWarps * kStages * kBatchBytes, "the bins take the stages' place");

__device__ __forceinline__ int pages_of(int tokens, int shift) { return tokens > 0 ? ((tokens - 1) >> shift) + 1 : 0; }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
// (nothing but that this CTA runs)
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// A word of shared memory of the cluster's CTA `rank`, at this CTA's address.
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t rank, uint32_t v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\t"
      "mapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.u32 [a], %2;\n\t}" ::"r"(addr), "r"(rank), "r"(v)
      : "memory");
}
// Asynchronous copies of this thread into shared memory; it alone reads them.
__device__ __forceinline__ void copy_16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_4(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {  // all but the last N groups
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t ld_l2(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.cg.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ int dp2a(uint32_t two16, uint32_t four8, int c, bool upper) {
  return upper ? __dp2a_hi(static_cast<int>(two16), static_cast<int>(four8), c)
               : __dp2a_lo(static_cast<int>(two16), static_cast<int>(four8), c);
}

// Larger-is-better order of scores as unsigned numbers; 0 is left for a page
// out of range.
__device__ __forceinline__ uint32_t score_key(float s) {
  const uint32_t u = __float_as_uint(s);
  return u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
}

// --------------------------------------------------------------------------
// Queries: up and down of a query token, in the order in which lanes use them
// --------------------------------------------------------------------------
constexpr int kQueryHeads = MLAQP_KV4_MAX_HEADS / kSelectHeadGroups;
struct QueryPart {
  uint32_t v[kQueryHeads][4];  // this thread's eight channels of its heads: pairs of BF16, or E4M3 codes in the first two
};

// Four E4M3 codes as FP16 pairs (exact; NaN stays one).
__device__ __forceinline__ uint2 e4m3x4_f16(uint32_t c) {
  uint2 r;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(r.x), "=r"(r.y)
      : "r"(c));
  return r;
}
__device__ __forceinline__ float f16_lo(uint32_t v) {
  float f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.f32.f16 %0, a;\n\t}" : "=f"(f) : "r"(v));
  return f;
}
__device__ __forceinline__ float f16_hi(uint32_t v) { return f16_lo(v >> 16); }

template <bool E4>
__device__ __forceinline__ void load_query(const Kv4SelectParams& p, int64_t m, QueryPart& q) {
  const int chunk = threadIdx.x % kSelectChunks, g = threadIdx.x / kSelectChunks;
#pragma unroll
  for (int i = 0; i < kQueryHeads; ++i) {
    const int h = g + kSelectHeadGroups * i;
    uint32_t(&v)[4] = q.v[i];
    v[0] = v[1] = v[2] = v[3] = 0;
    if (h >= p.H) continue;
    const int64_t at = m * p.q_ts + h * kOutDim + 8 * chunk;
    if constexpr (E4) {
      asm volatile("ld.global.v2.b32 {%0,%1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "l"(p.q + at));
    } else {
      const uint4 w = ld_u128(reinterpret_cast<const uint16_t*>(p.q) + at);
      v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    }
  }
}

// Into `words` ([32 lanes][kScoreLane], this CTA's address) of `ctas` CTAs of
// the cluster, or of this one alone (0).  All threads call.
template <bool E4>
__device__ __forceinline__ void query_words(SelectShared& s, QueryPart& q, uint32_t* words, int ctas) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = tid % kSelectChunks, g = tid / kSelectChunks;
  uint32_t amax = 0;  // bits of the largest magnitude, BF16 or FP16
#pragma unroll
  for (int i = 0; i < kQueryHeads; ++i) {
    if constexpr (E4) {
      const uint2 x = e4m3x4_f16(q.v[i][0]), y = e4m3x4_f16(q.v[i][1]);
      q.v[i][0] = x.x, q.v[i][1] = x.y, q.v[i][2] = y.x, q.v[i][3] = y.y;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) amax = __vmaxu2(amax, q.v[i][u] & 0x7FFF7FFFu);
  }
  amax = __reduce_max_sync(0xffffffffu, max(amax & 0xFFFFu, amax >> 16));
  if (lane == 0) s.amax[warp] = amax;
  __syncthreads();  // (also: the token before has been read from s.part)
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) amax = max(amax, s.amax[w]);
  const bool none = amax >= (E4 ? 0x7C00u : 0x7F80u);  // a NaN or an infinity
  // 2047/1024 = 1 + 0x7FE000 * 2^-23
  const uint32_t top = __float_as_uint(E4 ? f16_lo(amax) : __uint_as_float(amax << 16));
  const int f = max(static_cast<int>((top + 0x1FFFu) >> 23) - 127 - 10, -100);
  const float scale = none ? 0.f : __uint_as_float(static_cast<uint32_t>(127 - f) << 23);
  // v + 1.5 * 2^23 rounds v to a whole number n, ties to even, and its bits are
  // those of 1.5 * 2^23 plus n: sums are of integers from there on.
  constexpr float kWhole = 12582912.f;
  constexpr int kWholeBits = 0x4B400000;
  int up[8] = {}, all[8] = {};
#pragma unroll
  for (int i = 0; i < kQueryHeads; ++i)
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t two = q.v[i][u >> 1];
      const float x = E4 ? (u & 1 ? f16_hi(two) : f16_lo(two)) : (u & 1 ? bf16_hi(two) : bf16_lo(two));
      const int n = __float_as_int(__fmaf_rn(x, scale, kWhole));
      all[u] += n - kWholeBits;
      up[u] += max(n, kWholeBits) - kWholeBits;
    }
  uint32_t packed[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) packed[u] = none ? 0u : static_cast<uint32_t>(up[u] << 16 | (up[u] - all[u]));
  *reinterpret_cast<uint4*>(&s.part[g][8 * chunk]) = make_uint4(packed[0], packed[1], packed[2], packed[3]);
  *reinterpret_cast<uint4*>(&s.part[g][8 * chunk + 4]) = make_uint4(packed[4], packed[5], packed[6], packed[7]);
  __syncthreads();
  // word w of lane l: pairs of up for the latents 16l.., of down for the same,
  // and of up (l < 16) or down for four rope elements
#pragma unroll
  for (int i = tid; i < 32 * kScoreWords; i += kSelectThreads) {
    const int l = i / kScoreWords, w = i % kScoreWords;
    const bool rope = w >= 16, high = rope ? l < 16 : w < 8;
    const int c = rope ? kLatent + 4 * (l & 15) + 2 * (w - 16) : 16 * l + 2 * (w & 7);
    uint2 sum = make_uint2(0, 0);  // neither half overflows: 16 heads * 2047
#pragma unroll
    for (int a = 0; a < kSelectHeadGroups; ++a) {
      const uint2 x = *reinterpret_cast<const uint2*>(&s.part[a][c]);
      sum.x += x.x, sum.y += x.y;
    }
    const uint32_t two = high ? __byte_perm(sum.x, sum.y, 0x7632) : __vneg2(__byte_perm(sum.x, sum.y, 0x5410));
    if (ctas == 0) {
      words[l * kScoreLane + w] = two;
    } else {
      const uint32_t at = smem_u32(&words[l * kScoreLane + w]);
      for (int r = 0; r < ctas; ++r) st_cluster(at, r, two);
    }
  }
}

// --------------------------------------------------------------------------
// Scores of four pages at a time
// --------------------------------------------------------------------------

// A warp's copy of a digest's bounds into `to`, and its score from there.  A
// lane copies what it reads: 16 bytes of either bound of the latents, 4 of the
// rope part's.
__device__ __forceinline__ void copy_digest(uint32_t to, const uint8_t* d) {
  const int lane = threadIdx.x & 31;
  copy_16(to + 16 * lane, d + 16 * lane);
  copy_16(to + kLatent + 16 * lane, d + kLatent + 16 * lane);
  copy_4(to + 2 * kLatent + 4 * lane, d + 2 * kLatent + 4 * lane);
}

// Keys of the four pages at `batch` for the query token of `words`; exps and
// good of page `first + u` lie with that lane.  Lane u < 4 gets page u's.
__device__ __forceinline__ uint32_t score_batch(const uint8_t* batch, const uint32_t* words, uint32_t exps, bool good, int first) {
  const int lane = threadIdx.x & 31;
  const uint32_t* w = words + lane * kScoreLane;
  int a[kScorePages], r[kScorePages];
#pragma unroll
  for (int u = 0; u < kScorePages; ++u) a[u] = 0;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint4 x = *reinterpret_cast<const uint4*>(w + 8 * half), y = *reinterpret_cast<const uint4*>(w + 8 * half + 4);
#pragma unroll
    for (int u = 0; u < kScorePages; ++u) {
      const uint4 d = *reinterpret_cast<const uint4*>(batch + u * 2 * kOutDim + half * kLatent + 16 * lane);
      a[u] = dp2a(x.x, d.x, a[u], false), a[u] = dp2a(x.y, d.x, a[u], true);
      a[u] = dp2a(x.z, d.y, a[u], false), a[u] = dp2a(x.w, d.y, a[u], true);
      a[u] = dp2a(y.x, d.z, a[u], false), a[u] = dp2a(y.y, d.z, a[u], true);
      a[u] = dp2a(y.z, d.w, a[u], false), a[u] = dp2a(y.w, d.w, a[u], true);
    }
  }
  const uint2 z = *reinterpret_cast<const uint2*>(w + 16);
#pragma unroll
  for (int u = 0; u < kScorePages; ++u) {
    const uint32_t d = *reinterpret_cast<const uint32_t*>(batch + u * 2 * kOutDim + 2 * kLatent + 4 * lane);
    r[u] = __reduce_add_sync(0xffffffffu, dp2a(z.y, d, dp2a(z.x, d, 0, false), true));
    a[u] = __reduce_add_sync(0xffffffffu, a[u]);
  }
  // from here on a page a lane
  const int u = lane & (kScorePages - 1);
  const int sum = u & 2 ? (u & 1 ? a[3] : a[2]) : (u & 1 ? a[1] : a[0]);
  const int rsum = u & 2 ? (u & 1 ? r[3] : r[2]) : (u & 1 ? r[1] : r[0]);
  exps = __shfl_sync(0xffffffffu, exps, first + u);
  good = __shfl_sync(0xffffffffu, static_cast<int>(good), first + u);
  const uint32_t ea = exps & 255u, er = exps >> 8 & 255u;
  float f = __fadd_rn(__fmul_rn(static_cast<float>(sum), __uint_as_float(ea << 23)),
                      __fmul_rn(static_cast<float>(rsum), __uint_as_float(er << 23)));
  if (ea == 255u || er == 255u) f = INFINITY;
  return good ? score_key(f) : 0u;
}

// --------------------------------------------------------------------------
// Choice of a query token's pages
// --------------------------------------------------------------------------

// Exclusive sums of two numbers over the CTA, in thread order (x, y), and their
// totals (z, w).  Not inlined: code that is run for the first time waits for
// its fetch.
__device__ __noinline__ int4 choose_scan(SelectShared& s, int a, int b) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = a, y = b;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, x, d), v = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) x += u, y += v;
  }
  __syncthreads();  // of an earlier call
  if (lane == 31) s.scan[warp][0] = x, s.scan[warp][1] = y;
  __syncthreads();
  int4 sum = make_int4(x - a, y - b, 0, 0);
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) {
    if (w < warp) sum.x += s.scan[w][0], sum.y += s.scan[w][1];
    sum.z += s.scan[w][0], sum.w += s.scan[w][1];
  }
  return sum;
}

// Query token m, which sees n tokens; row: its sequence's pages.  held: the
// place of its keys in s.keys, -1 where they are in the workspace.  All threads call.
__device__ __forceinline__ void choose_pages(const Kv4SelectParams& p, SelectShared& s, unsigned* bins, int m, int n,
                                             const int32_t* row, int held_at) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pages = pages_of(n, p.shift);
  const int taken = min(pages, p.k);
  int32_t* out = p.table + m * p.sel_stride;
  if (tid == 0) p.lens[m] = pages > 0 ? ((taken - 1) << p.shift) + (n - ((pages - 1) << p.shift)) : 0;
  for (int r = taken + tid; r < p.k; r += kSelectThreads) out[r] = -1;
  const bool held = held_at >= 0;
  auto page_at = [&](int j) { return held ? s.pages[j] : row[j]; };
  if (pages <= p.k) {
    for (int r = tid; r < pages; r += kSelectThreads) out[r] = page_at(r);
    return;
  }
  for (int r = tid; r < p.first + p.last; r += kSelectThreads)
    out[r < p.first ? r : p.k - p.last + (r - p.first)] = page_at(r < p.first ? r : pages - p.last + (r - p.first));
  const int keep = p.k - p.first - p.last, count = pages - p.first - p.last;  // of the pages between
  if (keep == 0) return;
  const uint32_t* far_keys = p.keys + m * p.width + p.first;
  auto key_of = [&](int j) { return held ? s.keys[held_at + j] : ld_l2(far_keys + j); };

  // the range of the keys
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
  __syncthreads();  // the bins of the token before, or the stages, are done with
  for (int j = tid; j < count; j += kSelectThreads) {
    const uint32_t key = key_of(j);
    lo = min(lo, key);
    hi = max(hi, key);
  }
  if (tid == 0) s.found = 0;
  for (int e = tid; e < kBins / 4; e += kSelectThreads) reinterpret_cast<uint4*>(bins)[e] = make_uint4(0, 0, 0, 0);
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) s.lo[warp] = lo, s.hi[warp] = hi;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSelectWarps; ++w) lo = min(lo, s.lo[w]), hi = max(hi, s.hi[w]);
  if (lo == 0 && tid == 0) atomicOr(&g_device_status, kDevStatusBadIndex);
  // Keys from `lo` to `hi`, `open` bits of them undecided: the place that holds
  // the last one taken, until all in it are taken or all in it are equal.
  int open = 32 - __clz(hi - lo), above = 0, in = count;
  while (open > 0 && above + in != keep) {
    const int drop = max(open - kBinsLog, 0);
    for (int j = tid; j < count; j += kSelectThreads) {
      const uint32_t key = key_of(j);
      if (key >= lo && key - lo <= hi - lo) atomicAdd(&bins[(key - lo) >> drop], 1u);
    }
    __syncthreads();
    // thread t: eight bins from the top, cleared for the next round
    unsigned here[kBinsEach] = {};
    int sum = 0;
    if (tid < kBinThreads) {
      uint4* at = reinterpret_cast<uint4*>(bins + kBins - kBinsEach * (tid + 1));
      const uint4 x = at[0], y = at[1];
      at[0] = at[1] = make_uint4(0, 0, 0, 0);
      here[0] = y.w, here[1] = y.z, here[2] = y.y, here[3] = y.x;
      here[4] = x.w, here[5] = x.z, here[6] = x.y, here[7] = x.x;
#pragma unroll
      for (int e = 0; e < kBinsEach; ++e) sum += here[e];
    }
    int before = above + choose_scan(s, sum, 0).x;
    if (before < keep && keep <= before + sum) {
#pragma unroll
      for (int e = 0; e < kBinsEach; ++e) {
        const int with = before + static_cast<int>(here[e]);
        if (before < keep && keep <= with) {
          s.from = lo + (static_cast<uint32_t>(kBins - 1 - (tid * kBinsEach + e)) << drop);
          s.above = before;
          s.in = here[e];
        }
        before = with;
      }
    }
    __syncthreads();
    lo = s.from;
    hi = lo + ((1u << drop) - 1u);
    above = s.above;
    in = s.in;
    open = drop;
    if (open > 0 && above + in != keep && in <= kCandidates) {
      // few are left: every warp ranks them
      for (int j = tid; j < count; j += kSelectThreads) {
        const uint32_t key = key_of(j);
        if (key >= lo && key <= hi) s.candidate[atomicAdd(&s.found, 1)] = key;
      }
      __syncthreads();
      const uint32_t mine = lane < in ? s.candidate[lane] : 0u;
      int more = 0, same = 0;
#pragma unroll 1
      for (int c = 0; c < in; ++c) {
        const uint32_t key = __shfl_sync(0xffffffffu, mine, c);
        more += key > mine;
        same += key == mine;
      }
      const bool last = lane < in && above + more < keep && keep <= above + more + same;
      const int who = __ffs(__ballot_sync(0xffffffffu, last)) - 1;
      lo = hi = __shfl_sync(0xffffffffu, mine, who);
      above += __shfl_sync(0xffffffffu, more, who);
      open = 0;
    }
  }
  // taken: keys above hi, and of those from lo to hi the first keep - above
  int done = 0, equal = 0;
  for (int j0 = 0; j0 < count; j0 += kSelectThreads * kChooseEach) {
    uint32_t key[kChooseEach];
    int a = 0, e = 0;
    const int j = j0 + tid * kChooseEach;
#pragma unroll
    for (int u = 0; u < kChooseEach; ++u) {
      key[u] = j + u < count ? key_of(j + u) : 0;
      if (j + u < count) a += key[u] > hi, e += key[u] >= lo && key[u] <= hi;
    }
    const int4 before = choose_scan(s, a, e);
    int nth = equal + before.y;
    int at = p.first + done + before.x + min(nth, keep - above);
#pragma unroll
    for (int u = 0; u < kChooseEach; ++u) {
      if (j + u >= count) break;
      const bool mid = key[u] >= lo && key[u] <= hi;
      if (key[u] > hi || (mid && nth < keep - above)) out[at++] = page_at(p.first + j + u);
      nth += mid;
    }
    done += before.z;
    equal += before.w;
  }
}

// --------------------------------------------------------------------------
// One cluster a sequence: queries, scores, choice
// --------------------------------------------------------------------------
template <bool E4>
__global__ void __launch_bounds__(kSelectThreads, kSelectCtasPerSm)
    mlaqp_kv4_select_kernel(const __grid_constant__ Kv4SelectParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  SelectShared& s = *reinterpret_cast<SelectShared*>(smem);
  uint32_t* const words = reinterpret_cast<uint32_t*>(smem + kWordsAt);  // [q_len][kQueryWords]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ctas = p.cluster, rank = static_cast<int>(cluster_rank());
  const int b = blockIdx.x / ctas;
  pdl_launch_dependents();
  if (ctas > 1) cluster_arrive_relaxed();
  pdl_wait();
  // Several query tokens are shared out: each CTA sees to some of them, for all.
  const bool share = ctas > 1 && p.q_len > 1;
  const int64_t m0 = static_cast<int64_t>(b) * p.q_len;
  const int step = share ? ctas : 1;
  int i = share ? rank : 0;
  QueryPart q;
  if (i < p.q_len) load_query<E4>(p, m0 + i, q);  // (where nothing is to be scored, for nothing)
  const int seq = p.seqs ? p.seqs[b] : b;
  bool bad = seq < 0 || seq >= p.num_seqs;
  int len = 0;
  if (!bad) {
    len = p.seq_lens[seq];
    bad = len < 0 || len > p.table_stride << p.shift || len > p.num_pages << p.shift;
  }
  if (bad) {
    if (tid == 0 && rank == 0) atomicOr(&g_device_status, kDevStatusBadIndex);
    len = 0;
  }
  const int32_t* row = p.block_table + (bad ? 0 : seq * p.table_stride);
  // pages to be scored: those between the first and the last ones of the last
  // query token, which sees the most
  const int pages = pages_of(len, p.shift);
  const int count = pages > p.k ? pages - p.first - p.last : 0;
  const int tokens = (p.q_len + ctas - 1) / ctas;  // a CTA chooses for tokens rank, rank + ctas, ..
  const bool held = count > 0 && pages <= kHeldKeys && static_cast<int64_t>(tokens) * count <= kHeldKeys;
  if (count > 0) {
    const int32_t* between = row + p.first;
    // Batch k of this warp is four entries, its lane u + 4 (k % 8) holding page
    // u: entries and exponents of eight batches at a time.
    const int warps = kSelectWarps * ctas, mine = kSelectWarps * rank + warp;
    const int batches = ((count + kScorePages - 1) / kScorePages - mine + warps - 1) / warps;
    auto entry = [&](int k0) {
      const int n = kScorePages * (warps * (k0 + lane / kScorePages) + mine) + lane % kScorePages;
      return n < count ? between[n] : -1;
    };
    auto digest_of = [&](int page) { return p.digests + page * p.digest_stride; };
    auto in_pool = [&](int page) { return page >= 0 && page < p.num_pages; };
    const uint32_t stages = smem_u32(smem + kStagesAt) + warp * kStages * kBatchBytes;
    auto copy_batch = [&](int k, int page) {  // page: of the eight batches with k
#pragma unroll
      for (int u = 0; u < kScorePages; ++u) {
        const int id = __shfl_sync(0xffffffffu, page, k % 8 * kScorePages + u);
        if (k < batches && in_pool(id)) copy_digest(stages + (k % kStages) * kBatchBytes + u * 2 * kOutDim, digest_of(id));
      }
      copy_commit();
    };
    int page = entry(0), next = -1;
    copy_batch(0, page);
    copy_batch(1, page);
    uint32_t exps = in_pool(page) ? ld_u32(digest_of(page) + 2 * kOutDim) : 0u, next_exps = 0;
    if (ctas > 1) cluster_wait();  // the others are there: their shared memory may be written
    for (; i < p.q_len; i += step) {
      query_words<E4>(s, q, words + i * kQueryWords, share ? ctas : 0);
      if (i + step < p.q_len) load_query<E4>(p, m0 + i + step, q);
    }
    if (share) {
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
    if (held && rank < p.q_len)  // for the choice, with whatever batch comes next
      for (int j = tid; j < pages; j += kSelectThreads) copy_4(smem_u32(&s.pages[j]), row + j);
#pragma unroll 1
    for (int k = 0; k < batches; ++k) {
      copy_wait<kStages - 1>();
      const uint8_t* batch = smem + kStagesAt + (warp * kStages + k % kStages) * kBatchBytes;
      const int at = k % 8 * kScorePages;
      const int n = kScorePages * (warps * k + mine) + lane;
#pragma unroll 1
      for (int t = 0; t < p.q_len; ++t) {
        const uint32_t key = score_batch(batch, words + t * kQueryWords, exps, in_pool(page), at);
        if (lane < kScorePages && n < count) {
          if (!held)
            p.keys[(m0 + t) * p.width + p.first + n] = key;
          else
            st_cluster(smem_u32(&s.keys[t / ctas * count + n]), t % ctas, key);
        }
      }
      // what comes next: a batch into this one's place, and its entries long before
      if (k % 8 == 0) next = entry(k + 8);
      if (k % 8 == 4) next_exps = in_pool(next) ? ld_u32(digest_of(next) + 2 * kOutDim) : 0u;
      copy_batch(k + kStages, k % 8 + kStages < 8 ? page : next);
      if (k % 8 == 7) page = next, exps = next_exps;
    }
    copy_wait<0>();
    if (ctas > 1) {  // all keys are there
      cluster_arrive();
      cluster_wait();
    } else {
      __syncthreads();
    }
  } else if (ctas > 1) {
    cluster_wait();
  }
  unsigned* bins = reinterpret_cast<unsigned*>(smem + kStagesAt);
  for (int t = rank; t < p.q_len; t += ctas)
    choose_pages(p, s, bins, static_cast<int>(m0) + t, max(0, len - (p.q_len - 1 - t)), row, held ? t / ctas * count : -1);
}


const void* select_kernel(bool e4m3) {
  return e4m3 ? reinterpret_cast<const void*>(&mlaqp_kv4_select_kernel<true>)
              : reinterpret_cast<const void*>(&mlaqp_kv4_select_kernel<false>);
}

constexpr size_t select_bytes(int q_len) { return kWordsAt + sizeof(uint32_t) * kQueryWords * static_cast<size_t>(q_len); }

}  // namespace

cudaError_t kv4_select(const Kv4SelectParams& params, bool q_e4m3, int sm_count, cudaStream_t stream) {
  Kv4SelectParams p = params;
  p.cluster = kSelectMaxCluster;
  while (p.cluster > 1 && p.B * p.cluster > kSelectCtasPerSm * sm_count) p.cluster /= 2;
  const int64_t some = (p.width + kSelectWarps * kScorePages - 1) / (kSelectWarps * kScorePages);
  while (p.cluster > 1 && p.cluster / 2 >= some) p.cluster /= 2;
  void* args[1] = {&p};
  return kv4_launch(select_kernel(q_e4m3), static_cast<unsigned>(p.B * p.cluster), kSelectThreads, select_bytes(p.q_len),
                    stream, args, static_cast<unsigned>(p.cluster));
}

cudaError_t kv4_select_setup() {
  cudaFuncAttributes a;
  cudaError_t e = cudaSuccess;
  for (const void* k : {select_kernel(false), select_kernel(true)}) {
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(select_bytes(MLAQP_KV4_MAX_Q_LEN)));
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, k);
  }
  return e;
}

cudaError_t device_status_kv4_select(unsigned int* value, bool reset) { return read_device_status(value, reset); }

}  // namespace mlaqp
